// short_conv.hip -- short causal convolution, one filter of K = 2 .. 4 taps for
// each channel, with SiLU or without: forward, backward and decode step.
//
//   u_t = b + sum_j w_j x_{t-K+1+j},  y_t = act(u_t)
// and with g_t = dy_t act'(u_t):
//   dx_s = sum_j w_j g_{s+K-1-j},  dw_j = sum_t g_t x_{t-K+1+j},  db = sum_t g_t.
//
// HBM-bound: x is read and y written once (backward: x, dy, dx).  A thread owns
// a piece of four channels and walks down a slab of rows with the last
// K - 1 rows (and, in the backward, the last K - 1 g) in registers, so that every
// row is loaded once but for the K - 1 rows around a slab, and four rows' loads of
// whole pieces are in flight while four are worked on (each load is a branch on the
// piece being whole; the rows ahead of a slab, which may be the state's, are waited
// for one after the other); LPR threads cover a row's piece of channels and the
// workgroup's other threads other slabs.  y (and
// dy) is head-major, the layout of the attentions: the transposition is an
// address.  The weights' gradients stay in registers down the slab, are summed
// over the workgroup's slabs through LDS, and leave one part for each workgroup
// (at most kMostParts), which a second kernel adds in a fixed order.
//
// MI355X, B4 T4096 C2048 K4 bf16 with SiLU: forward 33 us (4.1 TB/s of 134 MB), backward
// 67 (62 and 5 for the parts' sums; 3.0 TB/s of 201 MB); fp32 69 and 102 (3.9 and 4.0
// TB/s).  The backward in bf16 has the vector units busy for two thirds of its time
// (164 registers, three waves on a SIMD) and still no unit full;
// shorter slabs, slabs that fill the SIMDs exactly once, an order of the workgroups by
// L2 and an inner loop without the masks (177 registers instead of 164) gave nothing or
// lost.  Decode, 256 sequences of 4096 channels: a kernel of 7.4 us for 17 MB (3.4 at the
// copy's rate): a thread's sequences go one after the other, each one's loads behind the
// stores of the one before.
#include <limits.h>

#include <algorithm>

#include "ckda_internal.hpp"
#include "row_vec.hpp"

namespace ckda {

namespace {

constexpr int kConvThreads = 256;
constexpr int kMostParts = 1024;
constexpr int kUnroll = 4;   // rows whose loads are in flight together

struct ConvGeom {
  int B, T, C, H, Dh, ldx;
  int lpr;         // threads along the channels (a power of two)
  int cblocks;     // workgroups along the channels
  int rows;        // rows of a thread's slab
  int slabs;       // slabs of a workgroup's rows in a sequence
  int items;       // B slabs
  int parts;       // workgroups along the items
  int pad_zero;
};

// Rows of a thread's slab: longer slabs read less twice, shorter ones fill the
// CUs; by the pieces of 512 channels, so that the sums' parts do not depend on
// how the channels can be read.
int conv_rows(int B, int T, int C) {
  const double pieces = (double)B * ((C + 511) / 512);   // (of sizes that are refused too)
  int rows = 32;
  while (rows > 4 && pieces * ((T + rows - 1) / rows) < 2048) rows /= 2;
  return rows;
}

// Weights of a thread's channels: K VEC floats next to each other (16-byte loads: one by one they would be as
// many loads as a slab has rows).
template <int VEC, int K> struct ConvTaps {
  float w[K][VEC], b[VEC];
  __device__ __forceinline__ void load(const float* wp, const float* bp, int c0, int left) {
    float raw[K * VEC];
    wp += (size_t)c0 * K;
    if (VEC > 1 && left >= VEC) {
#pragma unroll
      for (int i = 0; i < K * VEC; i += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(wp + i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < K * VEC) raw[i + e] = v[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < K * VEC; ++i) raw[i] = i < left * K ? wp[i] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
      for (int j = 0; j < K; ++j) w[j][e] = raw[e * K + j];
    }
    if (!bp) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = 0.f;
    } else if (VEC > 1 && left >= VEC) {
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(bp + c0 + e);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < VEC) b[e + i] = v[i];
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = e < left ? bp[c0 + e] : 0.f;
    }
  }
};

// row t of a sequence: of x, or for t < 0 of the state before it
template <typename T, int VEC, int K>
__device__ __forceinline__ void load_row(RowVec<T, VEC>& v, const T* xb, const T* sb, int t, int ldx, int C, int left) {
  if (t >= 0) v.load(xb + (size_t)t * ldx, left);
  else if (sb) v.load(sb + (size_t)(t + K - 1) * C, left);
  else v.clear();
}

template <typename T, int VEC, int K, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_fwd_kernel(const T* x, const float* w, const float* b, const T* s0,
                                                                const int* lens, T* y, T* sT, ConvGeom G) {
  const int tx = threadIdx.x & (G.lpr - 1), sub = threadIdx.x / G.lpr, nsub = kConvThreads / G.lpr;
  const int cb = blockIdx.x % G.cblocks, item = blockIdx.x / G.cblocks;
  const int batch = item / G.slabs, slab = item - batch * G.slabs;
  const int c0 = (cb * G.lpr + tx) * VEC, left = G.C - c0;
  if (left <= 0) return;
  const int len = lens ? min(max(lens[batch], 0), G.T) : G.T;
  const long long first = ((long long)slab * nsub + sub) * G.rows;
  const T* xb = x + (size_t)batch * G.T * G.ldx + c0;
  const T* sb = s0 ? s0 + (size_t)batch * (K - 1) * G.C + c0 : nullptr;
  if (slab == 0 && sub == 0 && sT) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      RowVec<T, VEC> v;
      load_row<T, VEC, K>(v, xb, sb, len - (K - 1) + i, G.ldx, G.C, left);
      v.store(sT + ((size_t)batch * (K - 1) + i) * G.C + c0, left);
    }
  }
  if (first >= G.T) return;
  const int r0 = (int)first, r1 = min(r0 + G.rows, G.T), live = min(r1, len);
  const int h = c0 / G.Dh;
  T* yb = y + ((size_t)batch * G.H + h) * G.T * G.Dh + (c0 - h * G.Dh);
  if (r0 < live) {
    ConvTaps<VEC, K> taps;
    taps.load(w, b, c0, left);
    float win[K - 1 + kUnroll][VEC];
    {
      RowVec<T, VEC> v[K - 1];
#pragma unroll
      for (int i = 0; i < K - 1; ++i) load_row<T, VEC, K>(v[i], xb, sb, r0 - (K - 1) + i, G.ldx, G.C, left);
#pragma unroll
      for (int i = 0; i < K - 1; ++i) v[i].widen(win[i]);
    }
    RowVec<T, VEC> v[kUnroll];
    // rows behind the slab: its last row once more (no branch on the row, so that whole pieces' loads stay in flight)
    auto fetch = [&](int t) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u].load(xb + (size_t)min(t + u, live - 1) * G.ldx, left);
    };
    fetch(r0);
    for (int t = r0; t < live; t += kUnroll) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) v[u].widen(win[K - 1 + u]);
      fetch(t + kUnroll);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float a = taps.b[e];
#pragma unroll
          for (int j = 0; j < K; ++j) a = __builtin_fmaf(taps.w[j][e], win[u + j][e], a);
          o[e] = SILU ? a * row_sigmoid<T>(a) : a;
        }
        RowVec<T, VEC> q;
        q.round(o);
        if (t + u < live) q.store(yb + (size_t)(t + u) * G.Dh, left);
      }
#pragma unroll
      for (int i = 0; i < K - 1; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) win[i][e] = win[kUnroll + i][e];
    }
  }
  if (G.pad_zero) {
    RowVec<T, VEC> v;
    v.clear();
    for (int t = max(r0, live); t < r1; ++t) v.store(yb + (size_t)t * G.Dh, left);
  }
}

template <typename T, int VEC, int K, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_bwd_kernel(const T* x, const float* w, const float* b, const T* s0,
                                                                const int* lens, const T* dy, const T* dsT, T* dx, T* ds0,
                                                                float* part, ConvGeom G) {
  const int tx = threadIdx.x & (G.lpr - 1), sub = threadIdx.x / G.lpr, nsub = kConvThreads / G.lpr;
  const int cb = blockIdx.x % G.cblocks, p = blockIdx.x / G.cblocks;
  const int c0 = (cb * G.lpr + tx) * VEC, left = G.C - c0;
  ConvTaps<VEC, K> taps;
  taps.load(w, b, c0, left);
  float dw[K][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = 0.f;
  }
  const int h = left > 0 ? c0 / G.Dh : 0;
  for (int item = p; item < G.items && left > 0; item += G.parts) {
    const int batch = item / G.slabs, slab = item - batch * G.slabs;
    const long long first = ((long long)slab * nsub + sub) * G.rows;
    if (first >= G.T && first > 0) continue;   // (without any row the first slab still makes ds0)
    const int len = lens ? min(max(lens[batch], 0), G.T) : G.T;
    const int r0 = (int)first, r1 = min(r0 + G.rows, G.T);
    const T* xb = x + (size_t)batch * G.T * G.ldx + c0;
    const T* sb = s0 ? s0 + (size_t)batch * (K - 1) * G.C + c0 : nullptr;
    const T* gb = dy + ((size_t)batch * G.H + h) * G.T * G.Dh + (c0 - h * G.Dh);
    T* dxb = dx + (size_t)batch * G.T * G.C + c0;
    float win[K - 1 + kUnroll][VEC], gw[K - 1 + kUnroll][VEC];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      RowVec<T, VEC> v;
      if (r0 - (K - 1) + i < len) load_row<T, VEC, K>(v, xb, sb, r0 - (K - 1) + i, G.ldx, G.C, left);
      else v.clear();
      v.widen(win[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) gw[i][e] = 0.f;
    }
    // row t makes g_t, and with it dx_{t-K+1}; of the slab's last K - 1 rows by the rows behind it
    RowVec<T, VEC> v[kUnroll], q[kUnroll];
    const int last = min(len, r1 + K - 1) - 1;
    // rows behind the last one: that one once more, masked below
    auto fetch = [&](int t) {
      if (last < r0) return;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        v[u].load(xb + (size_t)min(t + u, last) * G.ldx, left);
        q[u].load(gb + (size_t)min(t + u, last) * G.Dh, left);
      }
    };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u].clear(), q[u].clear();
    fetch(r0);
    for (int t = r0; t < r1 + K - 1; t += kUnroll) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        v[u].widen(win[K - 1 + u]);
        q[u].widen(gw[K - 1 + u]);
      }
      fetch(t + kUnroll);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float* g = gw[K - 1 + u];
        const bool live = t + u < len && t + u < r1 + K - 1, mine = live && t + u < r1;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if constexpr (SILU) {
            float a = taps.b[e];
#pragma unroll
            for (int j = 0; j < K; ++j) a = __builtin_fmaf(taps.w[j][e], win[u + j][e], a);
            g[e] *= silu_slope(a, row_sigmoid<T>(a));
          }
          g[e] = live ? g[e] : 0.f;
          const float own = mine ? g[e] : 0.f;
          db[e] += own;
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j][e] = __builtin_fmaf(own, win[u + j][e], dw[j][e]);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int s = t + u - (K - 1);
        if (s >= r1 || (s < r0 && r0 > 0)) continue;
        float d[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          d[e] = 0.f;
#pragma unroll
          for (int i = 0; i < K; ++i) d[e] = __builtin_fmaf(taps.w[K - 1 - i][e], gw[u + i][e], d[e]);
        }
        const int at_end = s - (len - (K - 1));   // row of the final state that this input is
        if (dsT && at_end >= 0 && at_end < K - 1) {
          RowVec<T, VEC> f;
          f.load(dsT + ((size_t)batch * (K - 1) + at_end) * G.C + c0, left);
          float fv[VEC];
          f.widen(fv);
#pragma unroll
          for (int e = 0; e < VEC; ++e) d[e] += fv[e];
        }
        RowVec<T, VEC> o;
        o.round(d);
        if (s < 0) {
          if (ds0) o.store(ds0 + ((size_t)batch * (K - 1) + s + K - 1) * G.C + c0, left);
        } else if (s < len || G.pad_zero) {
          o.store(dxb + (size_t)s * G.C, left);
        }
      }
#pragma unroll
      for (int i = 0; i < K - 1; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          win[i][e] = win[kUnroll + i][e];
          gw[i][e] = gw[kUnroll + i][e];
        }
    }
  }
  if (!part) return;
  // the workgroup's sums over its slabs; a part is [C, K] then [C]
  __shared__ float s_sum[kConvThreads * VEC];
  float* to = part + (size_t)p * G.C * (K + 1);
  const int cols = G.lpr * VEC, cbase = cb * cols;
#pragma unroll
  for (int q = 0; q <= K; ++q) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) s_sum[(sub * G.lpr + tx) * VEC + e] = q < K ? dw[q < K ? q : 0][e] : db[e];
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += kConvThreads) {
      if (cbase + c >= G.C) break;
      float a = 0.f;
      for (int i = 0; i < nsub; ++i) a += s_sum[i * cols + c];
      if (q < K) to[(size_t)(cbase + c) * K + q] = a;
      else to[(size_t)G.C * K + cbase + c] = a;
    }
  }
}

// A thread owns a piece of channels of `each` sequences (the weights are read once).
template <typename T, int VEC, int K, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_decode_kernel(const T* x, const float* w, const float* b, T* state,
                                                                   T* y, int N, int C, int pieces, int ldx, int each) {
  const long long i = (long long)blockIdx.x * kConvThreads + threadIdx.x;
  const long long first = i / pieces * each;
  const int c0 = (int)(i % pieces) * VEC, left = C - c0;
  if (first >= N) return;
  ConvTaps<VEC, K> taps;
  taps.load(w, b, c0, left);
  for (int m = 0; m < each && first + m < N; ++m) {
    const size_t n = first + m;
    RowVec<T, VEC> v[K];
    T* sb = state + n * (K - 1) * C + c0;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) v[j].load(sb + (size_t)j * C, left);
    v[K - 1].load(x + n * ldx + c0, left);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) v[j + 1].store(sb + (size_t)j * C, left);
    float o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = taps.b[e];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float r[VEC];
      v[j].widen(r);
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = __builtin_fmaf(taps.w[j][e], r[e], o[e]);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = SILU ? o[e] * row_sigmoid<T>(o[e]) : o[e];
    v[0].round(o);
    v[0].store(y + n * C + c0, left);
  }
}

ConvGeom conv_geom(const ShortConvArgs& a, int vec) {
  ConvGeom G;
  G.B = a.B, G.T = a.T, G.C = a.C, G.H = a.H, G.Dh = a.C / a.H, G.ldx = a.ldx, G.pad_zero = a.pad_zero;
  const int pieces = (a.C + vec - 1) / vec;
  G.lpr = 1;
  while (G.lpr < 64 && G.lpr < pieces) G.lpr *= 2;
  G.cblocks = (pieces + G.lpr - 1) / G.lpr;
  G.rows = conv_rows(a.B, a.T, a.C);
  const long long per = (long long)G.rows * (kConvThreads / G.lpr);
  G.slabs = (int)std::max(1LL, (a.T + per - 1) / per);
  G.items = a.B * G.slabs;
  G.parts = std::min(G.items, kMostParts);
  return G;
}

enum class ConvOp { fwd, bwd, decode };

template <ConvOp OP, typename T, int VEC, int K, bool SILU> hipError_t launch_conv_t(const ShortConvArgs& a) {
  if constexpr (OP == ConvOp::decode) {
    const int pieces = (a.C + VEC - 1) / VEC;
    const int each = (int)std::max(1LL, std::min(4LL, (long long)a.B * pieces / 65536));
    const long long blocks = (((long long)a.B + each - 1) / each * pieces + kConvThreads - 1) / kConvThreads;
    hipLaunchKernelGGL((conv_decode_kernel<T, VEC, K, SILU>), dim3((unsigned)blocks), dim3(kConvThreads), 0, a.stream,
                       (const T*)a.x, a.w, a.b, (T*)a.state, (T*)a.y, a.B, a.C, pieces, a.ldx, each);
    return hipGetLastError();
  } else {
    const ConvGeom G = conv_geom(a, VEC);
    if constexpr (OP == ConvOp::fwd) {
      hipLaunchKernelGGL((conv_fwd_kernel<T, VEC, K, SILU>), dim3((unsigned)G.items * G.cblocks), dim3(kConvThreads), 0,
                         a.stream, (const T*)a.x, a.w, a.b, (const T*)a.s0, a.lens, (T*)a.y, (T*)a.sT, G);
      return hipGetLastError();
    }
    const bool weights = a.dw || a.db;
    if (G.items > 0) {
      hipLaunchKernelGGL((conv_bwd_kernel<T, VEC, K, SILU>), dim3((unsigned)G.parts * G.cblocks), dim3(kConvThreads), 0,
                         a.stream, (const T*)a.x, a.w, a.b, (const T*)a.s0, a.lens, (const T*)a.dy, (const T*)a.dsT, (T*)a.dx,
                         (T*)a.ds0, weights ? (float*)a.workspace : nullptr, G);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess || !weights) return e;
    }
    const size_t C = (size_t)a.C;
    return launch_part_sums(PartSums{(const float*)a.workspace, G.parts, C * (K + 1), {a.dw, a.db, nullptr}, {C * K, C, 0}},
                            a.stream);
  }
}

template <ConvOp OP, typename T, int VEC> hipError_t launch_conv_v(const ShortConvArgs& a) {
  switch (a.K * 2 + (a.silu ? 1 : 0)) {
    case 4: return launch_conv_t<OP, T, VEC, 2, false>(a);
    case 5: return launch_conv_t<OP, T, VEC, 2, true>(a);
    case 6: return launch_conv_t<OP, T, VEC, 3, false>(a);
    case 7: return launch_conv_t<OP, T, VEC, 3, true>(a);
    case 8: return launch_conv_t<OP, T, VEC, 4, false>(a);
    case 9: return launch_conv_t<OP, T, VEC, 4, true>(a);
  }
  return hipErrorInvalidValue;
}

// Pieces of four channels (with bf16 8 bytes: half the registers of 16, so twice the waves; MI355X, us, four and
// eight: forward B4 T4096 C2048 31.5 and 39, backward 66 and 143), or single ones where a piece would lie across
// two heads.
template <ConvOp OP> hipError_t launch_conv(const ShortConvArgs& a) {
  const bool pieces = a.H == 1 || (a.C / a.H) % 4 == 0;
  if (a.dtype == CKDA_DTYPE_BF16) return pieces ? launch_conv_v<OP, bf16_t, 4>(a) : launch_conv_v<OP, bf16_t, 1>(a);
  return pieces ? launch_conv_v<OP, float, 4>(a) : launch_conv_v<OP, float, 1>(a);
}

}  // namespace

// the most parts a call leaves: those of one slab of rows a workgroup
size_t short_conv_bwd_workspace_bytes(int B, int T, int C, int K) {
  const long long rows = 4 * (long long)conv_rows(B, T, C);   // four slabs a workgroup at least
  const long long items = (long long)B * std::max(1LL, (T + rows - 1) / rows);
  return (size_t)std::min<long long>(items, kMostParts) * C * (K + 1) * 4;
}

// fewer than 2^24 workgroups of 256 threads, however the channels are read, and 2^22 of 1024 for the parts' sums
bool short_conv_fits_grid(int B, int T, int C, int H) {
  const long long rows = 4 * (long long)conv_rows(B, T, C), pieces = (C + 63) / 64;
  const long long slabs = std::max(1LL, (T + rows - 1) / rows);
  return (long long)B * slabs <= INT_MAX && (long long)B * slabs * pieces < (1LL << 24) && H > 0 &&
         (long long)C * 5 < (1LL << 26);
}

hipError_t launch_short_conv_fwd(const ShortConvArgs& a) { return launch_conv<ConvOp::fwd>(a); }
hipError_t launch_short_conv_bwd(const ShortConvArgs& a) { return launch_conv<ConvOp::bwd>(a); }
hipError_t launch_short_conv_decode(const ShortConvArgs& a) { return launch_conv<ConvOp::decode>(a); }

}  // namespace ckda
