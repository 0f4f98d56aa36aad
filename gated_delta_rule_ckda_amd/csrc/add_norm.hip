// add_norm.hip -- root-mean-square norm with the residual's addition, in the
// inputs' type or in 8 bits with scales, forward and backward.
//
//   r = x + res,  s = (mean r^2 + eps)^-1/2,  n = r s,  y = n w
//   q = e4m3(y / scale),  scale = max |y| / 448 over a row or 128 of its columns
// and with dn = dy w:
//   dr = dsum + s (dn - n mean(dn n)),  dw = sum over rows of dy n.
//
// HBM-bound: every tensor is read or written once.  LPR threads hold one row in
// registers (NV pieces of 16 bytes of x each, and the same columns of the other
// tensors), a row's sum of squares is a sum over its threads (DPP, and LDS for
// rows that take the whole workgroup), and so are the largest values of the
// 8-bit form: 128 columns are 16 threads (bf16) or 32 (fp32) next to each other.
// A thread group walks over rows, the next row's loads in flight while it works on
// this one; w stays in registers.  In the backward dw does too; a workgroup
// leaves one part and a second kernel adds them in a fixed order.  All arithmetic
// is fp32; y, the codes, sum and dr are rounded once, from unrounded values.
//
// MI355X, 16384 x 2048 bf16 with an fp32 residual: forward to 8 bits with the sum 89 us
// (4.2 TB/s of 370 MB; a copy of 2 GiB moves 4.9), backward 118 (114 and 4 for the parts'
// sums; 4.6 TB/s of 537 MB).  One row: 2.4 us, the rest of its 9 is the call.
#include <algorithm>

#include "ckda_internal.hpp"
#include "row_vec.hpp"

namespace ckda {

namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.f;

// Sum over the LPR threads of a row; 256 threads go through LDS, in one of two
// alternating buffers so that one barrier is enough.
template <int LPR> __device__ __forceinline__ float row_sum(float x, float (*s)[kThreads / 64], int& phase) {
  x = group_sum<(LPR < 64 ? LPR : 64)>(x);
  if constexpr (LPR > 64) {
    float* buf = s[phase];
    phase ^= 1;
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (buf[0] + buf[1]) + (buf[2] + buf[3]);
  }
  return x;
}

// Largest of |x| over N neighbouring lanes, as the bits of a float: with integers
// a NaN is the largest of all.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
template <int CTRL> __device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true));
}
template <int N> __device__ __forceinline__ uint32_t group_max(uint32_t x) {
  static_assert(N >= 8 && N <= 64, "group size");
  x = dpp_max<0xB1>(x);                             // quad_perm [1,0,3,2]
  x = dpp_max<0x4E>(x);                             // quad_perm [2,3,0,1]
  x = dpp_max<0x141>(x);                            // row_half_mirror
  if constexpr (N >= 16) x = dpp_max<0x140>(x);     // row_mirror
  if constexpr (N >= 32) x = max(x, (uint32_t)__shfl_xor((int)x, 16, 64));
  if constexpr (N >= 64) x = max(x, (uint32_t)__shfl_xor((int)x, 32, 64));
  return x;
}

// scale of a group with largest value `top`, and the factors that take y to the
// range of the codes: pre keeps the reciprocal of a tiny scale finite.
struct Quant {
  float scale, pre, inv;
};
__device__ __forceinline__ Quant quant_of(uint32_t top_bits) {
  const float top = __uint_as_float(top_bits);
  Quant q;
  q.scale = top / kE4m3Max;
  q.pre = top < 0x1p-90f ? 0x1p100f : 1.f;
  q.inv = kE4m3Max / (top * q.pre);
  if (q.scale == 0.f) q.scale = q.pre = q.inv = 1.f;
  return q;
}

template <int VEC> __device__ __forceinline__ void store_codes(uint8_t* p, const float* y, Quant q, int left) {
  uint32_t w[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = y[4 * i + e] * q.pre * q.inv;
    int t = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], t, true);
  }
  if (left >= VEC) {
    __builtin_memcpy(p, w, VEC);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < left) p[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

struct NormGeom {
  int R, D;
  int steps;    // rows a thread group walks over
  int group;    // columns of one scale: 128, or D
};

// T: type of x, y and their gradients; TR: type of the residual and the sum
template <typename T, typename TR, int LPR, int NV>
__global__ __launch_bounds__(kThreads) void add_norm_fwd_kernel(const T* x, const TR* res, const float* w, T* y,
                                                                uint8_t* q, float* scales, TR* sum, NormGeom G,
                                                                float eps) {
  constexpr int VEC = kVec<T>, GPW = kThreads / LPR;
  __shared__ float s_sum[2][kThreads / 64];
  __shared__ uint32_t s_top[2][kThreads / 64];
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, D = G.D;
  int phase = 0, top_phase = 0;
  float wv[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * LPR + lane) * VEC;
    RowVec<float, 4> f[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      if (w) f[i].load(w + c + 4 * i, D - c - 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) wv[v][4 * i + e] = w ? f[i].e[e] : 1.f;
    }
  }
  const long long base = (long long)blockIdx.x * GPW * G.steps;
  RowVec<T, VEC> xr[NV];
  RowVec<TR, VEC / (sizeof(TR) / sizeof(T))> rr[NV][sizeof(TR) / sizeof(T)];
  constexpr int RP = sizeof(TR) / sizeof(T), RV = VEC / RP;   // pieces of TR beside one of T
  auto fetch = [&](long long row) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * VEC, left = row < G.R ? D - c : 0;
      xr[v].load(x + row * D + c, left);
#pragma unroll
      for (int i = 0; i < RP; ++i) {
        if (res) rr[v][i].load(res + row * D + c + i * RV, left - i * RV);
        else rr[v][i].clear();
      }
    }
  };
  fetch(base + grp);
  for (int step = 0; step < G.steps; ++step) {   // the same trips for every thread of the workgroup
    const long long row = base + (long long)step * GPW + grp;
    if (base + (long long)step * GPW >= G.R) break;
    float r[NV][VEC], sq = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float t[VEC];
      xr[v].widen(r[v]);
#pragma unroll
      for (int i = 0; i < RP; ++i) rr[v][i].widen(t + i * RV);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (res) r[v][e] += t[e];
        sq = __builtin_fmaf(r[v][e], r[v][e], sq);
      }
    }
    if (step + 1 < G.steps) fetch(row + GPW);
    const bool live = row < G.R;
    if (sum && live) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * LPR + lane) * VEC;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          RowVec<TR, RV> o;
          o.round(r[v] + i * RV);
          o.store(sum + row * D + c + i * RV, D - c - i * RV);
        }
      }
    }
    sq = row_sum<LPR>(sq, s_sum, phase);
    const float rstd = 1.f / sqrtf(sq / (float)D + eps);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) r[v][e] = r[v][e] * rstd * wv[v][e];
    if (y && live) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * LPR + lane) * VEC;
        RowVec<T, VEC> o;
        o.round(r[v]);
        o.store(y + row * D + c, D - c);
      }
    }
    if (!q) continue;
    // columns past the row count as zero for the largest value (w is zero there, but 0 times a NaN is not)
    uint32_t top[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      top[v] = 0;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if ((v * LPR + lane) * VEC + e < D) top[v] = max(top[v], abs_bits(r[v][e]));
    }
    constexpr int GL = 128 / VEC;   // threads of 128 columns
    if (G.group == 128) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        top[v] = group_max<(LPR < GL ? LPR : GL)>(top[v]);
        const Quant f = quant_of(top[v]);
        const int c = (v * LPR + lane) * VEC;
        if (live) store_codes<VEC>(q + row * D + c, r[v], f, D - c);
        if (live && c < D && lane % GL == 0) scales[row * ((D + 127) / 128) + c / 128] = f.scale;
      }
    } else {
#pragma unroll
      for (int v = 1; v < NV; ++v) top[0] = max(top[0], top[v]);
      uint32_t t = group_max<(LPR < 64 ? LPR : 64)>(top[0]);
      if constexpr (LPR > 64) {
        uint32_t* buf = s_top[top_phase];
        top_phase ^= 1;
        if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = t;
        __syncthreads();
        t = max(max(buf[0], buf[1]), max(buf[2], buf[3]));
      }
      const Quant f = quant_of(t);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * LPR + lane) * VEC;
        if (live) store_codes<VEC>(q + row * D + c, r[v], f, D - c);
      }
      if (live && lane == 0) scales[row] = f.scale;
    }
  }
}

template <typename T, typename TR, int LPR, int NV>
__global__ __launch_bounds__(kThreads) void add_norm_bwd_kernel(const TR* sum, const float* w, const T* dy,
                                                                const TR* dsum, T* dx, TR* dres, float* part, NormGeom G,
                                                                float eps) {
  constexpr int VEC = kVec<T>, GPW = kThreads / LPR;
  constexpr int RP = sizeof(TR) / sizeof(T), RV = VEC / RP;
  __shared__ float s_sum[2][kThreads / 64];
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, D = G.D;
  int phase = 0;
  float wv[NV][VEC], dw[NV][VEC];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * LPR + lane) * VEC;
    RowVec<float, 4> f[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      if (w) f[i].load(w + c + 4 * i, D - c - 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        wv[v][4 * i + e] = w ? f[i].e[e] : 1.f;
        dw[v][4 * i + e] = 0.f;
      }
    }
  }
  const long long base = (long long)blockIdx.x * GPW * G.steps;
  RowVec<T, VEC> gr[NV];
  RowVec<TR, RV> sr[NV][RP], dr[NV][RP];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * VEC, left = row < G.R ? D - c : 0;
      gr[v].load(dy + row * D + c, left);
#pragma unroll
      for (int i = 0; i < RP; ++i) {
        sr[v][i].load(sum + row * D + c + i * RV, left - i * RV);
        if (dsum) dr[v][i].load(dsum + row * D + c + i * RV, left - i * RV);
        else dr[v][i].clear();
      }
    }
  };
  fetch(base + grp);
  for (int step = 0; step < G.steps; ++step) {   // the same trips for every thread of the workgroup
    const long long row = base + (long long)step * GPW + grp;
    if (base + (long long)step * GPW >= G.R) break;
    float r[NV][VEC], g[NV][VEC], more[NV][VEC], sq = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      gr[v].widen(g[v]);
#pragma unroll
      for (int i = 0; i < RP; ++i) {
        sr[v][i].widen(r[v] + i * RV);
        dr[v][i].widen(more[v] + i * RV);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) sq = __builtin_fmaf(r[v][e], r[v][e], sq);
    }
    if (step + 1 < G.steps) fetch(row + GPW);
    sq = row_sum<LPR>(sq, s_sum, phase);
    const float rstd = 1.f / sqrtf(sq / (float)D + eps);
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        r[v][e] *= rstd;                                                  // n
        dw[v][e] = __builtin_fmaf(g[v][e], r[v][e], dw[v][e]);
        g[v][e] *= wv[v][e];                                              // dn
        dot = __builtin_fmaf(g[v][e], r[v][e], dot);
      }
    dot = row_sum<LPR>(dot, s_sum, phase) / (float)D;
    if (row >= G.R) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        r[v][e] = __builtin_fmaf(rstd, __builtin_fmaf(-r[v][e], dot, g[v][e]), more[v][e]);
      if (dx) {
        RowVec<T, VEC> o;
        o.round(r[v]);
        o.store(dx + row * D + c, D - c);
      }
      if (dres) {
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          RowVec<TR, RV> o;
          o.round(r[v] + i * RV);
          o.store(dres + row * D + c + i * RV, D - c - i * RV);
        }
      }
    }
  }
  if (!part) return;
  float* to = part + (size_t)blockIdx.x * D;
  if constexpr (GPW == 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (v * LPR + lane) * VEC + e;
        if (c < D) to[c] = dw[v][e];
      }
  } else {
    // sums over the workgroup's rows, one piece of columns after the other
    __shared__ float s_part[kThreads * VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) s_part[threadIdx.x * VEC + e] = dw[v][e];
      __syncthreads();
      for (int c = threadIdx.x; c < LPR * VEC; c += kThreads) {
        float a = 0.f;
#pragma unroll 4
        for (int i = 0; i < GPW; ++i) a += s_part[i * LPR * VEC + c];
        const int at = v * LPR * VEC + c;
        if (at < D) to[at] = a;
      }
    }
  }
}

struct NormShape {
  int lpr, nv;
};
// A wave for a row of up to 128 pieces, beyond that the workgroup: a wave of four pieces a lane has half the waves
// on a SIMD (MI355X, us, workgroup and wave: forward 16384 x 2048 bf16 51.5 and 71.5, in 8 bits with an fp32 residual
// 92 and 100, backward 120 and 131; 4096 x 1024 fp32 backward 19.4 and 21.4).
NormShape norm_shape(int D, int vec) {
  const int pieces = (D + vec - 1) / vec;
  NormShape s{8, 1};
  while (s.lpr < 64 && s.lpr < pieces) s.lpr *= 2;
  if (pieces > 128) s.lpr = 256;
  while (s.lpr * s.nv < pieces) s.nv *= 2;
  return s;
}

// Rows a thread group walks over: as many as leave the CUs 2048 workgroups
// (backward: 1024, which each leave a part).
int norm_steps(int R, int lpr, bool bwd) {
  const long long groups = (bwd ? 1024LL : 2048LL) * (kThreads / lpr);
  return (int)std::max(1LL, (R + groups - 1) / groups);
}

template <typename T, typename TR, int LPR, int NV> hipError_t launch_norm_t(const AddNormArgs& a, bool bwd) {
  const int per = kThreads / LPR;
  const NormGeom G{a.R, a.D, norm_steps(a.R, LPR, bwd), a.group ? a.group : a.D};
  const long long rows = (long long)per * G.steps;
  const unsigned blocks = (unsigned)((a.R + rows - 1) / rows);
  if (!bwd) {
    hipLaunchKernelGGL((add_norm_fwd_kernel<T, TR, LPR, NV>), dim3(blocks), dim3(kThreads), 0, a.stream, (const T*)a.x,
                       (const TR*)a.res, a.w, (T*)a.y, (uint8_t*)a.q, a.scales, (TR*)a.sum, G, a.eps);
    return hipGetLastError();
  }
  if (blocks > 0) {
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, TR, LPR, NV>), dim3(blocks), dim3(kThreads), 0, a.stream,
                       (const TR*)a.sum, a.w, (const T*)a.dy, (const TR*)a.dsum, (T*)a.dx, (TR*)a.dres,
                       a.dw ? (float*)a.workspace : nullptr, G, a.eps);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_part_sums(PartSums{(const float*)a.workspace, (int)blocks, (size_t)a.D, {a.dw, nullptr, nullptr},
                                   {(size_t)a.D, 0, 0}}, a.stream);
}

template <typename T, typename TR> hipError_t launch_norm_r(const AddNormArgs& a, bool bwd) {
  const NormShape s = norm_shape(a.D, kVec<T>);
  switch (s.lpr * 16 + s.nv) {
    case 8 * 16 + 1: return launch_norm_t<T, TR, 8, 1>(a, bwd);
    case 16 * 16 + 1: return launch_norm_t<T, TR, 16, 1>(a, bwd);
    case 32 * 16 + 1: return launch_norm_t<T, TR, 32, 1>(a, bwd);
    case 64 * 16 + 1: return launch_norm_t<T, TR, 64, 1>(a, bwd);
    case 64 * 16 + 2: return launch_norm_t<T, TR, 64, 2>(a, bwd);
    case 256 * 16 + 1: return launch_norm_t<T, TR, 256, 1>(a, bwd);
    case 256 * 16 + 2: return launch_norm_t<T, TR, 256, 2>(a, bwd);
    case 256 * 16 + 4: return launch_norm_t<T, TR, 256, 4>(a, bwd);
    case 256 * 16 + 8:
      if constexpr (sizeof(T) == 4) return launch_norm_t<T, TR, 256, 8>(a, bwd);
      break;
  }
  return hipErrorInvalidValue;
}

hipError_t launch_norm(const AddNormArgs& a, bool bwd) {
  if (a.dtype == CKDA_DTYPE_F32) return launch_norm_r<float, float>(a, bwd);
  return a.res_dtype == CKDA_DTYPE_F32 ? launch_norm_r<bf16_t, float>(a, bwd) : launch_norm_r<bf16_t, bf16_t>(a, bwd);
}

}  // namespace

size_t add_norm_bwd_workspace_bytes(int R, int D, int dtype) {
  const NormShape s = norm_shape(D, dtype == CKDA_DTYPE_BF16 ? kVec<bf16_t> : kVec<float>);
  const long long rows = (long long)(kThreads / s.lpr) * norm_steps(R, s.lpr, true);
  return (size_t)((R + rows - 1) / rows) * D * 4;
}

hipError_t launch_add_norm_fwd(const AddNormArgs& a) { return launch_norm(a, false); }
hipError_t launch_add_norm_bwd(const AddNormArgs& a) { return launch_norm(a, true); }

}  // namespace ckda
