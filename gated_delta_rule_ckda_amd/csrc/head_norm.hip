// head_norm.hip -- the norm that follows the attention: layer norm (or root
// mean square norm) of each head's output row with an optional output gate,
// forward and backward.
//
//   n = (x - m) s,  m = mean x (0 for the rms norm),  s = (mean (x - m)^2 + eps)^-1/2
//   y = (n w + b) act(z),   act = silu or sigmoid of the gate z (1 without)
// and with u = dy act(z), dn = u w:
//   dx = s (dn - mean dn - n mean(dn n))   (rms norm: without mean dn)
//   dz = dy (n w + b) act'(z),   dw = sum u n,   db = sum u  (over batch and time).
// x is head-major [B, H, T, D] as the attention writes it; z, y, dy and dz are
// token-major [B, T, H, D], the rows a projection reads or writes: the
// transposition between the two costs nothing here, where every row is
// touched once anyway.
//
// HBM-bound: every tensor is read or written once.  LPR lanes hold one row in
// registers (NV vectors of VEC elements each, 16 bytes but for odd bf16 widths),
// so the row's sums (mean, centred square sum, and in the backward the two
// means of dn) are DPP sums over the lane group (over the workgroup for rows
// of more than 64 x 4 vectors).  The statistics are recomputed in the backward
// from x, which it reads anyway, instead of being stored by the forward.  A
// workgroup keeps to one head and walks a slab of its rows, so that w and b
// are loaded once and dw and db stay in registers; a slab's sums go to the
// workspace and a second kernel adds the slabs in a fixed order.
// All arithmetic is fp32; only y, dx and dz are rounded, once.
#include <algorithm>

#include "ckda_device.hpp"
#include "ckda_internal.hpp"

namespace ckda {

namespace {

constexpr int kNormThreads = 256;
constexpr int kActNone = 0, kActSilu = CKDA_NORM_GATE_SILU, kActSigmoid = CKDA_NORM_GATE_SIGMOID;

// 16 bytes at a 4-byte boundary (global memory takes these at full width)
typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(4)));

// VEC consecutive elements (16 bytes, or one element): as loaded, and widened.
// `left` is how many of them the row still has: a row's last vector may be short.
template <typename T, int VEC> struct Vec {
  u32x4 w;
  __device__ __forceinline__ void load(const T* p, int left) {
    if (left >= VEC) {
      w = *reinterpret_cast<const u32x4a*>(p);
    } else {
      const uint32_t* d = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = i * VEC / 4 < left ? d[i] : 0u;
    }
  }
  __device__ __forceinline__ void clear() { w = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void widen(float* v) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo_half(w[i]);
        v[2 * i + 1] = bf16_hi_half(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
};
template <typename T> struct Vec<T, 1> {
  T w;
  __device__ __forceinline__ void load(const T* p, int) { w = *p; }
  __device__ __forceinline__ void clear() { w = from_f32<T>(0.f); }
  __device__ __forceinline__ void widen(float* v) const { v[0] = to_f32(w); }
};
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* v, int left) {
  if constexpr (VEC == 1) {
    *p = from_f32<T>(v[0]);
  } else {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      else w[i] = __float_as_uint(v[i]);
    }
    if (left >= VEC) {
      *reinterpret_cast<u32x4a*>(p) = w;
    } else {
      uint32_t* d = reinterpret_cast<uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i * VEC / 4 < left) d[i] = w[i];
    }
  }
}

// sigmoid(z).  With bf16 outputs by the hardware's exp2 and reciprocal (a few
// 2^-23, against an output rounding of 2^-8): the library's exponential and
// division are half of the backward's vector instructions, which then bound it.
template <typename T> __device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 2)
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
  else return 1.f / (1.f + expf(-z));
}

// K sums at once over the LPR lanes of a row; 256 lanes (the workgroup) go
// through LDS, in one of two alternating buffers so that one barrier is enough.
constexpr int kMostSums = 8;
template <int LPR, int K>
__device__ __forceinline__ void row_sums(float (&x)[K], float (*s)[kMostSums][kNormThreads / 64], int& phase) {
  static_assert(K <= kMostSums, "sums at once");
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = group_sum<(LPR < 64 ? LPR : 64)>(x[k]);
  if constexpr (LPR > 64) {
    float(*buf)[kNormThreads / 64] = s[phase];
    phase ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) buf[k][threadIdx.x >> 6] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = (buf[k][0] + buf[k][1]) + (buf[k][2] + buf[k][3]);
  }
}

// Rows of one lane group whose loads are in flight together.
constexpr int rows_in_flight(int n, bool bwd) { return n <= 8 ? (bwd ? 2 : 4) : 1; }

struct RowGeom {
  int H, T, D, rows, slab_rows;   // rows = B T of one head
  int heads_first;                // order of the workgroups
};

// Workgroups of all heads of one slab next to each other, so that the pieces
// of a token-major row are touched at about the same time.  MI355X, cold
// inputs, us, slabs first -> heads first:
//   forward   bf16 B4 H16 T4096 D128 55 -> 48, B4 H8 T4096 D256 53 -> 45, B2 H8 T4096 D512 47.5 -> 46;
//             fp32 B4 H16 T4096 D64 52 -> 41, B1 H32 T4096 D128 49 -> 41
//   backward  bf16 B4 H16 T4096 D128 86 -> 81, B1 H64 T4096 D128 83 -> 77, B4 H8 T4096 D256 87 -> 77;
//             fp32 B2 H8 T4096 D128 40 -> 34.5
// but, in the backward, for rows of 512 bytes and more in token-major rows of
// 8 KB and more (as measured; why these differ is not known):
//             bf16 B2 H8 T4096 D512 75 -> 82; fp32 B2 H16 T4096 D128 68 -> 78, B1 H32 T4096 D128 70 -> 76
bool heads_first(int H, int D, int es, bool bwd) { return !bwd || D * es < 512 || H * D * es < 8192; }

template <typename T, int VEC, int LPR, int NV, bool BWD>
__global__ __launch_bounds__(kNormThreads) void head_norm_kernel(const T* x, const T* z, const T* dy, const float* w,
                                                                 const float* b, T* out, T* dz, float* part,
                                                                 RowGeom G, int w_shared, int act, int rms, float eps) {
  constexpr int GPW = kNormThreads / LPR;   // rows in flight per workgroup
  constexpr int N = NV * VEC;
  constexpr int U = rows_in_flight(N, BWD);
  __shared__ float s_sum[LPR > 64 ? 2 : 1][kMostSums][kNormThreads / 64];
  const int tid = threadIdx.x, lane = tid % LPR, grp = tid / LPR;
  const int h = G.heads_first ? blockIdx.x : blockIdx.y;
  const int slab = G.heads_first ? blockIdx.y : blockIdx.x;
  const int row0 = slab * G.slab_rows;
  const int row1 = min(row0 + G.slab_rows, G.rows);
  const int D = G.D;
  const float inv_d = 1.f / (float)D;
  int phase = 0;

  float wv[N], bv[N];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = (v * LPR + lane) * VEC + e;
      const int at = (w_shared ? 0 : h * D) + c;
      wv[v * VEC + e] = c >= D ? 0.f : w ? w[at] : 1.f;
      bv[v * VEC + e] = c < D && b ? b[at] : 0.f;
    }
  float dw[BWD ? N : 1], db[BWD ? N : 1];
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] = db[i] = 0.f;
  }

  for (int base = row0; base < row1; base += U * GPW) {   // the same trips for every lane of the workgroup
    // the loads of U rows first
    Vec<T, VEC> xr[U][NV], zr[U][NV], gr[U][BWD ? NV : 1];
    bool live[U];
    size_t xo[U], yo[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = base + u * GPW + grp;
      live[u] = n < row1;
      const int bi = (live[u] ? n : row0) / G.T, t = (live[u] ? n : row0) - bi * G.T;
      xo[u] = (((size_t)bi * G.H + h) * G.T + t) * D;   // head-major row
      yo[u] = (((size_t)bi * G.T + t) * G.H + h) * D;   // token-major row
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * LPR + lane) * VEC;
        xr[u][v].clear();
        zr[u][v].clear();
        if constexpr (BWD) gr[u][v].clear();
        if (live[u] && c < D) {
          xr[u][v].load(x + xo[u] + c, D - c);
          if (act) zr[u][v].load(z + yo[u] + c, D - c);
          if constexpr (BWD) gr[u][v].load(dy + yo[u] + c, D - c);
        }
      }
    }
    float xv[U][N], mean[U], sq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mean[u] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) xr[u][v].widen(xv[u] + v * VEC);
#pragma unroll
      for (int i = 0; i < N; ++i) mean[u] += xv[u][i];
    }
    if (!rms) row_sums<LPR>(mean, s_sum, phase);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mean[u] = rms ? 0.f : mean[u] * inv_d;
      sq[u] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int i = v * VEC + e;
          xv[u][i] = (v * LPR + lane) * VEC + e < D ? xv[u][i] - mean[u] : 0.f;
          sq[u] = __builtin_fmaf(xv[u][i], xv[u][i], sq[u]);
        }
    }
    row_sums<LPR>(sq, s_sum, phase);
    float rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) rstd[u] = 1.f / sqrtf(sq[u] * inv_d + eps);
    if constexpr (!BWD) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float zv[N];
#pragma unroll
        for (int v = 0; v < NV; ++v) zr[u][v].widen(zv + v * VEC);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float y = __builtin_fmaf(xv[u][i] * rstd[u], wv[i], bv[i]);
          if (act) {
            const float sg = sigmoid<T>(zv[i]);
            y *= act == kActSilu ? zv[i] * sg : sg;
          }
          xv[u][i] = y;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = (v * LPR + lane) * VEC;
          if (live[u] && c < D) store_vec<T, VEC>(out + yo[u] + c, xv[u] + v * VEC, D - c);
        }
      }
    } else {
      float gv[U][N], m[2 * U];   // dn; its sum and that of dn n
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float zv[N];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          zr[u][v].widen(zv + v * VEC);
          gr[u][v].widen(gv[u] + v * VEC);
        }
        m[u] = m[U + u] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float nn = xv[u][i] * rstd[u];
          float f = gv[u][i];
          if (act) {
            const float sg = sigmoid<T>(zv[i]);
            const float slope = act == kActSilu ? sg * __builtin_fmaf(zv[i], 1.f - sg, 1.f) : sg * (1.f - sg);
            f *= act == kActSilu ? zv[i] * sg : sg;
            zv[i] = gv[u][i] * __builtin_fmaf(nn, wv[i], bv[i]) * slope;   // dz
          }
          dw[i] = __builtin_fmaf(f, nn, dw[i]);
          db[i] += f;
          xv[u][i] = nn;
          gv[u][i] = f * wv[i];
          m[u] += gv[u][i];
          m[U + u] = __builtin_fmaf(gv[u][i], nn, m[U + u]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = (v * LPR + lane) * VEC;
          if (live[u] && c < D && act) store_vec<T, VEC>(dz + yo[u] + c, zv + v * VEC, D - c);
        }
      }
      row_sums<LPR>(m, s_sum, phase);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float m1 = rms ? 0.f : m[u] * inv_d, m2 = m[U + u] * inv_d;
#pragma unroll
        for (int i = 0; i < N; ++i) xv[u][i] = rstd[u] * (gv[u][i] - m1 - xv[u][i] * m2);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = (v * LPR + lane) * VEC;
          if (live[u] && c < D) store_vec<T, VEC>(out + xo[u] + c, xv[u] + v * VEC, D - c);
        }
      }
    }
  }

  if constexpr (BWD) {
    // the workgroup's sums: over the lane groups of a wave, then over the waves
    constexpr int WAVES = kNormThreads / 64;
    constexpr int COLS = (LPR < 64 ? LPR : 64) * N;   // columns one wave holds
    __shared__ float s_part[LPR <= 64 ? WAVES : 1][LPR <= 64 ? COLS : 1];
    float* to = part + ((size_t)h * (G.heads_first ? gridDim.y : gridDim.x) + slab) * 2 * D;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float* acc = which ? db : dw;
      if constexpr (LPR <= 64) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int off = LPR; off < 64; off <<= 1) acc[i] += __shfl_xor(acc[i], off, 64);
        __syncthreads();
        if ((tid & 63) < LPR) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s_part[tid >> 6][(v * LPR + lane) * VEC + e] = acc[v * VEC + e];
        }
        __syncthreads();
        for (int c = tid; c < D; c += kNormThreads)
          to[which * D + c] = (s_part[0][c] + s_part[1][c]) + (s_part[2][c] + s_part[3][c]);
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const int c = (v * LPR + lane) * VEC + e;
            if (c < D) to[which * D + c] = acc[v * VEC + e];
          }
      }
    }
  }
}

// dw and db: the sums of the slabs' parts [nparts][2][D] of one weight head.
// 16 columns per workgroup, 64 threads on each.
constexpr int kRedCols = 16, kRedRows = 64;
__global__ __launch_bounds__(kRedCols * kRedRows) void norm_weight_grad_kernel(const float* part, int nparts, int D,
                                                                               float* dw, float* db) {
  __shared__ float s[kRedRows][kRedCols + 1];
  const int tid = threadIdx.x, c = blockIdx.x * kRedCols + tid % kRedCols, j = tid / kRedCols;
  const int which = blockIdx.y, head = blockIdx.z;
  const float* p = part + (size_t)head * nparts * 2 * D + (size_t)which * D;
  float x = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int i = j; i < nparts; i += kRedRows) x += p[(size_t)i * 2 * D + c];
  }
  s[j][tid % kRedCols] = x;
  __syncthreads();
  for (int half = kRedRows / 2; half > 0; half >>= 1) {
    if (j < half) s[j][tid % kRedCols] += s[j + half][tid % kRedCols];
    __syncthreads();
  }
  float* out = which ? db : dw;
  if (j == 0 && c < D && out) out[(size_t)head * D + c] = s[0][tid];
}

// lanes and vectors per row for width D (VEC elements per vector)
struct NormShape {
  int vec, lpr, nv;
};
NormShape norm_shape(int D, int dtype) {
  const int full = dtype == CKDA_DTYPE_BF16 ? 8 : 4;
  NormShape s;
  s.vec = D * (dtype == CKDA_DTYPE_BF16 ? 2 : 4) % 4 == 0 ? full : 1;   // rows of whole 4-byte words, else single elements
  const int pieces = (D + s.vec - 1) / s.vec;
  if (pieces <= 64) {
    s.lpr = 2;
    while (s.lpr < pieces) s.lpr *= 2;
    s.nv = 1;
    if (s.vec == 1 && s.lpr < 16) s.lpr = 16;
  } else if (pieces <= 256) {
    s.lpr = 64;
    s.nv = pieces <= 128 ? 2 : 4;
  } else {
    s.lpr = 256;
    s.nv = 2;
    while (s.nv * 256 < pieces) s.nv *= 2;
  }
  return s;
}

// rows of one head per workgroup: at least four per lane group, and at most
// about 4096 workgroups (fp32 B2 H16 T4096 D128, forward: 40 us, 47 with 2048;
// bf16 alike), or 1024 in the backward, whose slabs each leave a part (bf16 B4
// H16 T4096 D128: 76 us, 81 with 2048, 77 with 4096; fp32 68.5, 68.5 and 73)
int slab_rows(int rows, int H, int lpr, bool bwd) {
  const int gpw = kNormThreads / lpr;
  const long long most = std::max(1, (bwd ? 1024 : 4096) / H);
  const long long unit = 4LL * gpw;
  const long long need = (rows + most - 1) / most;
  return (int)std::max(unit, (need + unit - 1) / unit * unit);
}

template <typename T, int VEC, int LPR, int NV>
hipError_t launch_norm_t(const HeadNormArgs& a, bool bwd) {
  const int rows = a.H > 0 ? a.B * a.T : 0;
  RowGeom G{a.H, a.T, a.D, rows, slab_rows(rows, std::max(a.H, 1), LPR, bwd), heads_first(a.H, a.D, (int)sizeof(T), bwd)};
  const unsigned slabs = (G.rows + G.slab_rows - 1) / G.slab_rows;   // at most 4096
  const dim3 grid = G.heads_first ? dim3(a.H, slabs) : dim3(slabs, a.H);
  const int act = a.z ? a.flags & (kActSilu | kActSigmoid) : kActNone;
  const int rms = (a.flags & CKDA_NORM_RMS) ? 1 : 0, shared = a.wheads == 1;
  if (G.rows == 0)
    ;   // nothing but the weights' gradients, which are then zero
  else if (bwd)
    hipLaunchKernelGGL((head_norm_kernel<T, VEC, LPR, NV, true>), grid, dim3(kNormThreads), 0, a.stream, (const T*)a.x,
                       (const T*)a.z, (const T*)a.dy, a.w, a.b, (T*)a.dx, (T*)a.dz, (float*)a.workspace, G, shared, act,
                       rms, a.eps);
  else
    hipLaunchKernelGGL((head_norm_kernel<T, VEC, LPR, NV, false>), grid, dim3(kNormThreads), 0, a.stream, (const T*)a.x,
                       (const T*)a.z, (const T*)nullptr, a.w, a.b, (T*)a.y, (T*)nullptr, (float*)nullptr, G, shared, act,
                       rms, a.eps);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !bwd || (!a.dw && !a.db)) return e;
  // shared weights: the parts of all heads are one list
  const int nparts = (int)slabs * (shared ? a.H : 1);
  hipLaunchKernelGGL(norm_weight_grad_kernel, dim3((a.D + kRedCols - 1) / kRedCols, 2, a.wheads),
                     dim3(kRedCols * kRedRows), 0, a.stream, (const float*)a.workspace, nparts, a.D, a.dw, a.db);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t launch_norm_v(const HeadNormArgs& a, const NormShape& s, bool bwd) {
  if (s.lpr == 256) {
    switch (s.nv) {
      case 2: return launch_norm_t<T, VEC, 256, 2>(a, bwd);
      case 4: return launch_norm_t<T, VEC, 256, 4>(a, bwd);
      case 8:
        if constexpr (VEC * sizeof(T) <= 16 && (VEC == 1 || sizeof(T) == 4)) return launch_norm_t<T, VEC, 256, 8>(a, bwd);
        break;
      case 16:
        if constexpr (VEC == 1) return launch_norm_t<T, VEC, 256, 16>(a, bwd);
        break;
      case 32:
        if constexpr (VEC == 1) return launch_norm_t<T, VEC, 256, 32>(a, bwd);
        break;
    }
    return hipErrorInvalidValue;
  }
  if (s.nv == 4) return launch_norm_t<T, VEC, 64, 4>(a, bwd);
  if (s.nv == 2) return launch_norm_t<T, VEC, 64, 2>(a, bwd);
  switch (s.lpr) {
    case 2:
      if constexpr (VEC > 1) return launch_norm_t<T, VEC, 2, 1>(a, bwd);
      break;
    case 4:
      if constexpr (VEC > 1) return launch_norm_t<T, VEC, 4, 1>(a, bwd);
      break;
    case 8:
      if constexpr (VEC > 1) return launch_norm_t<T, VEC, 8, 1>(a, bwd);
      break;
    case 16: return launch_norm_t<T, VEC, 16, 1>(a, bwd);
    case 32: return launch_norm_t<T, VEC, 32, 1>(a, bwd);
    case 64: return launch_norm_t<T, VEC, 64, 1>(a, bwd);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_norm(const HeadNormArgs& a, bool bwd) {
  const NormShape s = norm_shape(a.D, a.dtype);
  if (a.dtype == CKDA_DTYPE_BF16)
    return s.vec == 1 ? launch_norm_v<bf16_t, 1>(a, s, bwd) : launch_norm_v<bf16_t, 8>(a, s, bwd);
  return launch_norm_v<float, 4>(a, s, bwd);
}

}  // namespace

size_t head_norm_bwd_workspace_bytes(int B, int H, int T, int D, int wheads, int dtype) {
  (void)wheads;
  const long long rows = (long long)B * T;
  if (rows == 0 || H == 0) return 0;
  const int per = slab_rows((int)rows, H, norm_shape(D, dtype).lpr, true);
  return (size_t)((rows + per - 1) / per) * H * 2 * D * 4;
}

hipError_t launch_head_norm_fwd(const HeadNormArgs& a) { return launch_norm(a, false); }
hipError_t launch_head_norm_bwd(const HeadNormArgs& a) { return launch_norm(a, true); }

}  // namespace ckda
