// selective_scan.hip -- the selective scan: a diagonal recurrence whose decay
// differs for every channel c and state n, forward, backward and decode step.
//
//   d_t = softplus(dt_t + bias),  a_t[n] = exp(d_t A[n])
//   h_t[n] = a_t[n] h_{t-1}[n] + d_t x_t B_t[n],   s_t = sum_n C_t[n] h_t[n]
//   y_t = (s_t + D x_t) silu(z_t)
// and with ds = dy silu(z), R_t = a_{t+1} R_{t+1} + ds_t C_t (R behind the end: dhT):
//   u_t = sum_n R_t B_t,  q_t[n] = a_t R_t h_{t-1},  v_t = sum_n q_t A
//   dx = d u + D ds,  dd = x u + v,  dA = sum_t d q,  dD = sum_t ds x,
//   dB_t[n] = sum_c d x R,  dC_t[n] = sum_c ds h,  dz = dy (s + D x) silu'(z).
//
// Bound by vector instructions: for every (row, channel, state) two products, an
// exponential and two fused products, at about 22 cycles for 64 of them.  So the
// layout is one that leaves nothing else to do for each of them:
//  * A DPP row of 16 lanes is one channel, each lane a state (N > 16: NS = 2 or 4
//    states a lane), the state in a register, time down a loop.
//  * Rows go by chunks of 16.  What a row has for each channel (d, d x, ds) is
//    made once, by the lane of that row, and handed to the channel's 16 lanes by
//    the row broadcast of DPP, an operand modifier that costs no instruction.
//  * Sums over the states (s, u, v) are made for 16 rows at once: a transposing
//    reduction leaves row j's sum in lane j, 33 instructions for 16 sums instead
//    of 64, and what follows them is again done once for each row and channel.
//  * Sums over the channels (dB, dC) swap halves and quarters of a wave between
//    the two and between two rows (3 instructions a row), then go through LDS.
//  * A workgroup is 32 channels (8 waves), which share B_t and C_t in LDS, as
//    fp32; its rows of x, dt, z, dy and y are read and written by whole rows of
//    its channels and turned in LDS.
// Few channels and many rows: the sequence runs in segments.  A first pass makes
// each segment's own end state, a second joins them (a segment's decay is exp(A
// sum d), closed), the main pass starts from the joined states.  The backward
// needs the states in reverse: the forward pass stores them every 16 rows (of its
// segment, joined when read), and the backward recomputes 16 rows in registers.
#include <limits.h>

#include <algorithm>
#include <utility>

#include "ckda_internal.hpp"
#include "row_vec.hpp"

namespace ckda {

namespace {

constexpr int kRows = 16;       // rows of a chunk, and lanes of a channel
constexpr int kCh = 32;         // channels of a workgroup
constexpr int kScanThreads = kRows * kCh;
constexpr int kWaves = kScanThreads / 64;
// registers for two to four waves on a SIMD: rows' operands are loaded ahead, not one after the other
#define CKDA_SCAN_WAVES __attribute__((amdgpu_waves_per_eu(2, 4)))
constexpr int kPad = kRows + 1;   // row of a turned tile in LDS
constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = 1.9259629911266174e-8f, kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- lanes

template <int... J, typename F> __device__ __forceinline__ void each_impl(std::integer_sequence<int, J...>, F&& f) {
  (f(std::integral_constant<int, J>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F&& f) {
  each_impl(std::make_integer_sequence<int, N>{}, f);
}

// lane J's value of each DPP row, in all of its 16 lanes
template <int J> __device__ __forceinline__ float row_bcast(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + J, 0xF, 0xF, true));
}
template <int CTRL> __device__ __forceinline__ float dpp_mov(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// Sums over the 16 lanes of a DPP row of 16 values, value j's sum to lane j.  Each
// step pairs lanes across one bit of the lane number: a lane keeps the half of the
// values that has its bit and adds the partner's.  Where the bit selects whole
// banks of four lanes the second sum is written over the first under a bank mask
// (two instructions for two values), inside a bank it takes two selects and a sum.
// (The wait states a DPP source needs behind its writer stand in the asm itself.)
#define CKDA_PAIR(d, a, b, move, mask)                                      \
  "v_add_f32_dpp " d ", " a ", " a " " move " row_mask:0xf bank_mask:0xf\n" \
  "v_add_f32_dpp " d ", " b ", " b " " move " row_mask:0xf bank_mask:" mask "\n"
__device__ __forceinline__ float turn_sums(const float (&v)[kRows], int lane) {
  float a[8], b[4];
  asm("s_nop 1\n"   //
      CKDA_PAIR("%0", "%8", "%16", "row_ror:8", "0xc") CKDA_PAIR("%1", "%9", "%17", "row_ror:8", "0xc")
      CKDA_PAIR("%2", "%10", "%18", "row_ror:8", "0xc") CKDA_PAIR("%3", "%11", "%19", "row_ror:8", "0xc")
      CKDA_PAIR("%4", "%12", "%20", "row_ror:8", "0xc") CKDA_PAIR("%5", "%13", "%21", "row_ror:8", "0xc")
      CKDA_PAIR("%6", "%14", "%22", "row_ror:8", "0xc") CKDA_PAIR("%7", "%15", "%23", "row_ror:8", "0xc")
      : "=&v"(a[0]), "=&v"(a[1]), "=&v"(a[2]), "=&v"(a[3]), "=&v"(a[4]), "=&v"(a[5]), "=&v"(a[6]), "=&v"(a[7])
      : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]), "v"(v[8]), "v"(v[9]),
        "v"(v[10]), "v"(v[11]), "v"(v[12]), "v"(v[13]), "v"(v[14]), "v"(v[15]));
  asm("s_nop 1\n"   //
      CKDA_PAIR("%0", "%4", "%8", "row_half_mirror", "0xa") CKDA_PAIR("%1", "%5", "%9", "row_half_mirror", "0xa")
      CKDA_PAIR("%2", "%6", "%10", "row_half_mirror", "0xa") CKDA_PAIR("%3", "%7", "%11", "row_half_mirror", "0xa")
      : "=&v"(b[0]), "=&v"(b[1]), "=&v"(b[2]), "=&v"(b[3])
      : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(a[4]), "v"(a[5]), "v"(a[6]), "v"(a[7]));
  const bool two = lane & 2, one = lane & 1;
  const float c0 = (two ? b[2] : b[0]) + dpp_mov<0x4E>(two ? b[0] : b[2]);   // quad_perm [2,3,0,1]
  const float c1 = (two ? b[3] : b[1]) + dpp_mov<0x4E>(two ? b[1] : b[3]);
  return (one ? c1 : c0) + dpp_mov<0xB1>(one ? c0 : c1);                     // quad_perm [1,0,3,2]
}
#undef CKDA_PAIR

__device__ __forceinline__ void pin_float(float& x) { asm volatile("" : "+v"(x)); }

// lower half of the wave: a summed over the halves; upper half: b
__device__ __forceinline__ float sum_halves(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// even DPP rows: a summed over the row and the next; odd ones: b
__device__ __forceinline__ float sum_quarters(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ---------------------------------------------------------------- elements

// exp(-|v|), to a few 2^-24 (the product with log2 e in two parts)
__device__ __forceinline__ float exp_neg_abs(float v) {
  const float m = fminf(fabsf(v), 200.f), t = -m * kLog2e;
  const float lo = __builtin_fmaf(-m, kLog2eLo, __builtin_fmaf(-m, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, lo * kLn2, e);
}
// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|), by the series of log((1 +
// r) / (1 - r)) in r = e / (2 + e) <= 1/3 (next term 2^-26 of the first): small
// steps keep their relative accuracy, which log(1 + e) does not.
__device__ __forceinline__ float softplus(float v) {
  const float e = exp_neg_abs(v), r = e * __builtin_amdgcn_rcpf(2.f + e), z = r * r;
  float p = 1.f / 13.f;
  p = __builtin_fmaf(p, z, 1.f / 11.f);
  p = __builtin_fmaf(p, z, 1.f / 9.f);
  p = __builtin_fmaf(p, z, 1.f / 7.f);
  p = __builtin_fmaf(p, z, 1.f / 5.f);
  p = __builtin_fmaf(p, z, 1.f / 3.f);
  return (v < 0.f ? 0.f : v) + 2.f * __builtin_fmaf(r * z, p, r);   // (a NaN stays one)
}
__device__ __forceinline__ float softplus_slope(float v) {
  const float e = exp_neg_abs(v), r = __builtin_amdgcn_rcpf(1.f + e);
  return v >= 0.f ? r : e * r;
}

// A decay 2^x.  Where the inputs are bf16: itself, by the hardware's exponential
// (mean error -0.12 of 2^-24 for small x, so a state that remembers M rows is off
// by some 7e-9 M).  Where they are fp32: for -x < 1/16 its distance from 1, which
// keeps slow decays to 2^-24 of their rate (degree 4: next term 2^-25); stronger
// ones, of states that remember fewer than 24 rows, themselves.
template <bool EXACT> struct Decay;
template <> struct Decay<false> {
  float m;
  __device__ __forceinline__ explicit Decay(float x) : m(__builtin_amdgcn_exp2f(x)) {}
  __device__ __forceinline__ Decay() {}
  __device__ __forceinline__ float of(float h) const { return m * h; }
  __device__ __forceinline__ float of(float h, float add) const { return __builtin_fmaf(m, h, add); }
};
template <> struct Decay<true> {
  float m;
  bool near;   // m is the distance from 1
  __device__ __forceinline__ explicit Decay(float x) : near(fabsf(x) < 0.0625f) {
    float p = 0.009618129107628477f;                        // ln2^4 / 24
    p = __builtin_fmaf(p, x, 0.05550410866482158f);         // ln2^3 / 6
    p = __builtin_fmaf(p, x, 0.2402265069591007f);          // ln2^2 / 2
    p = __builtin_fmaf(p, x, kLn2);
    m = near ? p * x : __builtin_amdgcn_exp2f(x);
  }
  __device__ __forceinline__ Decay() {}
  __device__ __forceinline__ float of(float h) const { return __builtin_fmaf(m, h, near ? h : 0.f); }
  __device__ __forceinline__ float of(float h, float add) const { return __builtin_fmaf(m, h, add) + (near ? h : 0.f); }
};

// ---------------------------------------------------------------- launches

struct ScanGeom {
  int B, T, C, G, N;
  int Cg, cblocks;         // channels of a group, workgroups along them
  int ldbc, ldz;
  int nseg, seg_chunks;    // segments, chunks of each
  int chunks;              // chunks of T rows
  int softplus, pad_zero;
};

struct ScanWork {            // workspace of a call
  float* ends;               // [B][nseg][C][N]: segments' own end states, then start states
  float* steps;              // [B][nseg][C]: sums of d over the segments
  float* back;               // [B][nseg][C][N]: backward in time
  float* marks;              // [B][chunks][C][N]: states before each chunk, of their segment
  float* mark_steps;         // [B][chunks][C]: sums of d from the segment's start to each chunk (nseg > 1)
  float* bc;                 // [G cblocks][B T][2][N]: parts of dC, dB
  float* weights;            // [B nseg][C N + 2 C]: parts of dA, dD, dbias
};

struct ScanLaunch {
  SelScanArgs a;
  ScanGeom G;
  ScanWork w;
  int segs;                  // segments of this launch
};

// Place of a workgroup: the channel blocks of one piece of rows next to each
// other on one XCD, since they share lines of x, B and C.
struct ScanPlace {
  int b, seg, g, cb, len, ch0, ch1;
};
__device__ __forceinline__ bool scan_place(const ScanLaunch& L, ScanPlace& p) {
  const ScanGeom& G = L.G;
  const int total = G.B * L.segs * G.G * G.cblocks, per = (total + 7) / 8;
  int i = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (i >= total || (int)(blockIdx.x / 8) >= per) return false;
  p.cb = i % G.cblocks;
  i /= G.cblocks;
  p.g = i % G.G;
  i /= G.G;
  p.seg = i % L.segs;
  p.b = i / L.segs;
  p.len = L.a.lens ? min(max(L.a.lens[p.b], 0), G.T) : G.T;
  const int all = (p.len + kRows - 1) / kRows;
  p.ch0 = p.seg * G.seg_chunks;
  p.ch1 = min(p.ch0 + G.seg_chunks, all);
  return true;
}

// Rows of a tensor through a buffer resource that covers the rows of one tile: a
// thread's offset in the tile never changes, the resource moves (scalar registers),
// and rows behind the end and columns that are none (kNowhere) read zero and are not
// written, without a branch.
constexpr int kNowhere = 0x7FFFFFFF;
template <typename T> struct Rows {
  const char* base;      // first row of the segment
  uint32_t bytes;        // of a row
  __device__ __forceinline__ Rows(const void* p, size_t first, int ld)
      : base((const char*)p + first * ld * sizeof(T)), bytes((uint32_t)ld * sizeof(T)) {}
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t tile(int row, int rows) const {
    row = __builtin_amdgcn_readfirstlane(row), rows = __builtin_amdgcn_readfirstlane(rows);   // (scalar registers)
    return make_rsrc(base + (size_t)row * bytes, (uint32_t)max(rows, 0) * bytes);
  }
};
template <typename T> __device__ __forceinline__ uint32_t load_raw(__amdgpu_buffer_rsrc_t r, int off) {
  if constexpr (sizeof(T) == 2) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
  else return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}
template <typename T> __device__ __forceinline__ void store_elem(__amdgpu_buffer_rsrc_t r, int off, float x) {
  if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16((short)from_f32<bf16_t>(x).bits, r, off, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, off, 0, 0);
}
// A prefetched element, widened here and not where it was loaded (which would wait for it there).
template <typename T> __device__ __forceinline__ float value_of(uint32_t raw) {
  pin(raw);
  return __uint_as_float(sizeof(T) == 2 ? raw << 16 : raw);
}

// B and C (either alone: WHICH 1 or 2, both: 3) of SUBS chunks of rows in LDS, each
// as [row / 4][s][lane][row % 4], so that a lane reads four rows at once.  Every wave
// moves one of the two at a time.
template <typename T, int NS, int SUBS, int THREADS, int WHICH> struct BcTile {
  static constexpr int kOne = SUBS * kRows * 16 * NS;                  // elements of one of the two
  static constexpr int kEach = (WHICH == 3 ? 2 : 1) * kOne / THREADS;  // elements a thread moves
  static constexpr int kSpan = kOne < THREADS ? kOne : THREADS;        // threads on one of the two
  static constexpr int kLoads = kEach > 0 ? kEach : 1;
  uint32_t raw[kLoads];
  int off[kLoads];
  __device__ __forceinline__ static int place_of(int i) { return (int)threadIdx.x % kSpan + i % (kOne / kSpan) * kSpan; }
  __device__ __forceinline__ static bool of_c(int i) {
    if (WHICH != 3) return WHICH == 2;
    return kSpan < THREADS ? __builtin_amdgcn_readfirstlane((int)threadIdx.x) >= kSpan : i >= kOne / kSpan;
  }
  __device__ __forceinline__ static bool idle() { return WHICH != 3 && kSpan < THREADS && (int)threadIdx.x >= kSpan; }
  __device__ __forceinline__ void place(const ScanLaunch& L, const ScanPlace& p) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = place_of(i), n = idx % (16 * NS);
      off[i] = n < L.G.N && !idle() ? (idx / (16 * NS) * L.G.ldbc + p.g * L.G.N + n) * (int)sizeof(T) : kNowhere;
    }
  }
  __device__ __forceinline__ void fetch(const Rows<T>& B, const Rows<T>& C, int row, int rows) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      Rows<T> src = B;
      if (of_c(i)) src.base = C.base;
      raw[i] = load_raw<T>(src.tile(row, rows), off[i]);
    }
  }
  __device__ __forceinline__ void stage(float* s) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = place_of(i), n = idx % (16 * NS), row = idx / (16 * NS);
      if (!idle()) s[(of_c(i) && WHICH == 3 ? kOne : 0) + ((row / 4 * NS + n / 16) * 16 + n % 16) * 4 + row % 4] = value_of<T>(raw[i]);
    }
  }
};

// Block K of a tile's B or C: 16 / NS rows of NS states, f[row * NS + s].
template <int NS, int K> __device__ __forceinline__ void load_block(float (&f)[kRows], const float* one) {
  const f32x4* p = reinterpret_cast<const f32x4*>(one) + K * (4 / NS) * NS * 16 + (threadIdx.x & 15);
#pragma unroll
  for (int q = 0; q < 4 / NS; ++q)
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const f32x4 v = p[(q * NS + s) * 16];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[(4 * q + i) * NS + s] = v[i];
    }
}

// ---------------------------------------------------------------- forward

// MAIN: outputs (and the last state) from the segments' start states.  Else: the
// segments' own end states and sums of steps, with MARK the states before each
// chunk on the way (SEGS: of several segments).  Two chunks of rows between barriers.
template <typename T, int NS, int CH, bool MAIN, bool MARK, bool SEGS>
__global__ __launch_bounds__(kRows* CH) CKDA_SCAN_WAVES void scan_fwd_kernel(const ScanLaunch L) {
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int SUBS = 2, TILE = SUBS * kRows;
  __shared__ float2 s_d[2][SUBS][CH][kPad];
  __shared__ float s_y[MAIN ? 2 : 1][MAIN ? SUBS : 1][MAIN ? CH : 1][kPad];
  __shared__ __attribute__((aligned(16))) float s_bc[2][TILE * NS * 16 * (MAIN ? 2 : 1)];
  const SelScanArgs& a = L.a;
  const ScanGeom& G = L.G;
  ScanPlace p;
  if (!scan_place(L, p)) return;
  const int tid = threadIdx.x, n = tid & 15, mine = tid >> 4;   // state and channel in the recurrence
  const int r = tid / CH, ch = tid % CH;                         // row and channel of the tiles
  const int c0 = p.cb * CH, first_c = p.g * G.Cg + c0;
  const bool on = c0 + mine < G.Cg, tile_on = c0 + ch < G.Cg;
  const int cm = first_c + mine, ct = first_c + ch;
  const int row0 = p.ch0 * kRows, end = min(p.ch1 * kRows, p.len);   // rows of the segment

  float A2[NS], h[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const bool state = on && n + 16 * s < G.N;
    const size_t at = (size_t)cm * G.N + n + 16 * s;
    A2[s] = state ? a.A[at] * kLog2e : 0.f;
    h[s] = 0.f;
    if (state) {
      if (MAIN && p.seg > 0) h[s] = L.w.ends[((size_t)p.b * G.nseg + p.seg) * G.C * G.N + at];
      else if (p.seg == 0 && a.h0) h[s] = a.h0[(size_t)p.b * G.C * G.N + at];
    }
  }
  const float bias = tile_on && a.dt_bias ? a.dt_bias[ct] : 0.f;
  const float Dc = MAIN && tile_on && a.D ? a.D[ct] : 0.f;

  // this thread's rows of the tiles: row r, and every 16th from there
  const size_t first = (size_t)p.b * G.T + row0;
  const Rows<T> xs(a.x, first, G.C), ds(a.dt, first, G.C), ys(a.y, first, G.C), zs(a.z, first, G.ldz);
  const Rows<T> Bs(a.Bm, first, G.ldbc), Cs(a.Cm, first, G.ldbc);
  int off[SUBS], zoff[SUBS];
#pragma unroll
  for (int i = 0; i < SUBS; ++i) {
    off[i] = tile_on ? ((i * kRows + r) * G.C + ct) * (int)sizeof(T) : kNowhere;
    zoff[i] = tile_on ? ((i * kRows + r) * G.ldz + ct) * (int)sizeof(T) : kNowhere;
  }
  uint32_t xr[SUBS], dr[SUBS], zr[SUBS] = {};
  BcTile<T, NS, SUBS, kRows * CH, MAIN ? 3 : 1> bc;
  bc.place(L, p);
  // Rows behind the segment read zero; no branch around the loads (values that meet behind one are copied there,
  // and the copies wait for the loads).
  auto fetch = [&](int t0) {
    const int rows = min(end - t0, TILE), row = t0 - row0;
#pragma unroll
    for (int i = 0; i < SUBS; ++i) {
      xr[i] = load_raw<T>(xs.tile(row, rows), off[i]);
      dr[i] = load_raw<T>(ds.tile(row, rows), off[i]);
      if (MAIN) zr[i] = load_raw<T>(zs.tile(row, a.z ? rows : 0), zoff[i]);
    }
    bc.fetch(Bs, Cs, row, rows);
  };
  auto stage = [&](int buf, int t0) {
#pragma unroll
    for (int i = 0; i < SUBS; ++i) {
      float d = value_of<T>(dr[i]) + bias;
      if (G.softplus) d = softplus(d);
      d = tile_on && t0 + i * kRows + r < end ? d : 0.f;   // a step of zero leaves the state
      s_d[buf][i][ch][r] = float2{d, d * value_of<T>(xr[i])};
    }
    bc.stage(s_bc[buf]);
  };

  const Rows<float> marks(L.w.marks, (size_t)p.b * G.chunks, G.C * G.N), mark_sums(L.w.mark_steps, (size_t)p.b * G.chunks, G.C);
  int moff[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) moff[s] = on && n + 16 * s < G.N ? (cm * G.N + n + 16 * s) * 4 : kNowhere;

  float steps = 0.f;
  if (row0 < end) {
    fetch(row0);
    stage(0, row0);
    __syncthreads();
  }
  int buf = 0;
  for (int t0 = row0; t0 < end; t0 += TILE, buf ^= 1) {
    uint32_t xk[SUBS], zk[SUBS];
#pragma unroll
    for (int i = 0; i < SUBS; ++i) xk[i] = xr[i], zk[i] = zr[i];
    const bool more = t0 + TILE < end;
    fetch(t0 + TILE);
    // B and C of a block of rows are loaded while the block before is worked on
    const float* one = s_bc[buf];
    float2 d[SUBS];
    float Bv[2][kRows], Cv[2][kRows];
    load_block<NS, 0>(Bv[0], one);
    if constexpr (MAIN) load_block<NS, 0>(Cv[0], one + TILE * NS * 16);
#pragma unroll
    for (int i = 0; i < SUBS; ++i) d[i] = s_d[buf][i][mine][n];
    float sums[kRows];
    each<SUBS * NS>([&](auto K) {
      constexpr int k = K, i = k / NS, b = k % NS;   // block, its chunk and its place there
      if constexpr (k + 1 < SUBS * NS) {
        load_block<NS, k + 1>(Bv[(k + 1) % 2], one);
        if constexpr (MAIN) load_block<NS, k + 1>(Cv[(k + 1) % 2], one + TILE * NS * 16);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (b == 0) {
        if constexpr (MARK) {
          const int chunk = t0 / kRows + i;
#pragma unroll
          for (int s = 0; s < NS; ++s) store_elem<float>(marks.tile(chunk, chunk < p.ch1), moff[s], h[s]);
          if constexpr (SEGS) store_elem<float>(mark_sums.tile(chunk, chunk < p.ch1), on && n == 0 ? cm * 4 : kNowhere, steps);
        }
        if constexpr (SEGS) steps += group_sum<16>(d[i].x);
      }
      each<kRows / NS>([&](auto J) {
        constexpr int j = b * (kRows / NS) + J;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          h[s] = Decay<EXACT>(row_bcast<j>(d[i].x) * A2[s]).of(h[s], row_bcast<j>(d[i].y) * Bv[k % 2][J * NS + s]);
          if constexpr (MAIN) sums[j] = s ? __builtin_fmaf(Cv[k % 2][J * NS + s], h[s], sums[j]) : Cv[k % 2][J * NS] * h[s];
        }
      });
      if constexpr (MAIN && b == NS - 1) s_y[buf][i][mine][n] = turn_sums(sums, n);
    });
    if (more) stage(buf ^ 1, t0 + TILE);
    lds_barrier();
    if constexpr (MAIN) {
#pragma unroll
      for (int i = 0; i < SUBS; ++i) {
        float y = __builtin_fmaf(Dc, value_of<T>(xk[i]), s_y[buf][i][ch][r]);
        if (a.z) {
          const float z = value_of<T>(zk[i]);
          y *= z * row_sigmoid<T>(z);
        }
        store_elem<T>(ys.tile(t0 - row0, min(end - t0, TILE)), off[i], y);
      }
    }
  }
  if constexpr (MAIN) {
    if (a.hT && p.seg == G.nseg - 1 && on) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
        if (n + 16 * s < G.N) a.hT[((size_t)p.b * G.C + cm) * G.N + n + 16 * s] = h[s];
    }
    if (G.pad_zero && tile_on) {
      const int to = min((p.ch0 + G.seg_chunks) * kRows, G.T);
      for (int t = max(p.len, row0) + r; t < to; t += kRows) ((T*)a.y)[((size_t)p.b * G.T + t) * G.C + ct] = from_f32<T>(0.f);
    }
  } else if (SEGS && on) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (n + 16 * s < G.N) L.w.ends[(((size_t)p.b * G.nseg + p.seg) * G.C + cm) * G.N + n + 16 * s] = h[s];
    if (n == 0) L.w.steps[((size_t)p.b * G.nseg + p.seg) * G.C + cm] = steps;
  }
}

// Segments' own states joined in order, in place: each place gets the state that
// its segment starts from (forward in time: the first is left as it is, backward:
// the last).
template <bool EXACT, bool BACK> __global__ __launch_bounds__(256) void scan_join_kernel(const ScanLaunch L) {
  const ScanGeom& G = L.G;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, CN = (long long)G.C * G.N;
  if (i >= (long long)G.B * CN) return;
  const int b = (int)(i / CN);
  const long long cn = i - (long long)b * CN;
  const float A2 = L.a.A[cn] * kLog2e;
  float* own = (BACK ? L.w.back : L.w.ends) + (size_t)b * G.nseg * CN + cn;
  const float* steps = L.w.steps + (size_t)b * G.nseg * G.C + cn / G.N;
  float h = own[(size_t)(BACK ? G.nseg - 1 : 0) * CN];
  for (int k = 1; k < G.nseg; ++k) {
    const int seg = BACK ? G.nseg - 1 - k : k;
    // (the forward's launch of own states leaves out the last segment, whose end nobody starts from)
    const bool last = k == G.nseg - 1;
    const float next = last ? 0.f : own[(size_t)seg * CN], sum = last ? 0.f : steps[(size_t)seg * G.C];
    own[(size_t)seg * CN] = h;
    h = Decay<EXACT>(sum * A2).of(h) + next;
  }
}

// ---------------------------------------------------------------- backward

// MAIN: gradients.  Else: the segments' own states backward in time (the gradient
// of the state before a segment, from its rows alone).
template <typename T, int NS, bool MAIN, bool GATE>
__global__ __launch_bounds__(kScanThreads) CKDA_SCAN_WAVES void scan_bwd_kernel(const ScanLaunch L) {
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int kPartBufs = NS <= 2 ? 2 : 1;   // (two do not fit with 64 states)
  constexpr int kPart = kRows / 2 * NS * 64;   // a wave's dC and dB of a chunk: [row / 2][s][lane]
  __shared__ float2 s_d[2][kCh][kPad];
  __shared__ float s_ds[2][kCh][kPad];
  __shared__ float s_out[MAIN ? 2 : 1][3][MAIN ? kCh : 1][kPad];
  __shared__ __attribute__((aligned(16))) float s_bc[2][kRows * NS * 16 * (MAIN ? 2 : 1)];
  __shared__ __attribute__((aligned(16))) float s_part[MAIN ? kPartBufs : 1][MAIN ? kWaves : 1][MAIN ? kPart : 1];
  const SelScanArgs& a = L.a;
  const ScanGeom& G = L.G;
  ScanPlace p;
  if (!scan_place(L, p)) return;
  if (!MAIN) p.seg += 1, p.ch0 += G.seg_chunks, p.ch1 = min(p.ch0 + G.seg_chunks, (p.len + kRows - 1) / kRows);
  const int tid = threadIdx.x, n = tid & 15, mine = tid >> 4;
  const int r = tid / kCh, ch = tid % kCh;
  const int c0 = p.cb * kCh, first_c = p.g * G.Cg + c0;
  const bool on = c0 + mine < G.Cg, tile_on = c0 + ch < G.Cg;
  const int cm = first_c + mine, ct = first_c + ch;
  const size_t CN = (size_t)G.C * G.N;

  float A2[NS], A[NS], Q[NS], start[NS], dA[NS];
  bool state[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    state[s] = on && n + 16 * s < G.N;
    const size_t at = (size_t)cm * G.N + n + 16 * s;
    A[s] = state[s] ? a.A[at] : 0.f;
    A2[s] = A[s] * kLog2e;
    dA[s] = Q[s] = start[s] = 0.f;
    if (state[s]) {
      if (p.seg == G.nseg - 1) Q[s] = a.dhT ? a.dhT[(size_t)p.b * CN + at] : 0.f;
      else if (MAIN) Q[s] = L.w.back[((size_t)p.b * G.nseg + p.seg) * CN + at];
      if (MAIN && p.seg > 0) start[s] = L.w.ends[((size_t)p.b * G.nseg + p.seg) * CN + at];
    }
  }
  const float bias = tile_on && a.dt_bias ? a.dt_bias[ct] : 0.f;
  const float Dc = tile_on && a.D ? a.D[ct] : 0.f;
  float dD = 0.f, dbias = 0.f;

  const size_t first = (size_t)p.b * G.T;
  const Rows<T> xs(a.x, first, G.C), dts(a.dt, first, G.C), dys(a.dy, first, G.C), zs(a.z, first, G.ldz);
  const Rows<T> Bs(a.Bm, first, G.ldbc), Cs(a.Cm, first, G.ldbc);
  const Rows<T> dxs(a.dx, first, G.C), ddts(a.ddt, first, G.C), dzs(a.dz, first, G.C);
  const Rows<float> marks(L.w.marks, (size_t)p.b * G.chunks, G.C * G.N);
  const Rows<float> mark_sums(L.w.mark_steps, (size_t)p.b * G.chunks, G.C);
  const int off = tile_on ? (r * G.C + ct) * (int)sizeof(T) : kNowhere;
  const int zoff = tile_on ? (r * G.ldz + ct) * (int)sizeof(T) : kNowhere;
  uint32_t xr = 0, dr = 0, zr = 0, gr = 0, mark[NS], mark_steps = 0;
  BcTile<T, NS, 1, kScanThreads, MAIN ? 3 : 2> bc;
  bc.place(L, p);
  auto fetch = [&](int chunk) {   // (before the segment's first chunk: nothing; no branch around the loads)
    const int row = chunk * kRows, rows = chunk >= p.ch0 ? min(p.len - row, kRows) : 0;
    xr = load_raw<T>(xs.tile(row, MAIN ? rows : 0), off);
    dr = load_raw<T>(dts.tile(row, rows), off);
    gr = load_raw<T>(dys.tile(row, rows), off);
    zr = load_raw<T>(zs.tile(row, GATE ? rows : 0), zoff);
    bc.fetch(Bs, Cs, row, rows);
    if constexpr (MAIN) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
        mark[s] = load_raw<float>(marks.tile(chunk, rows > 0), state[s] ? (cm * G.N + n + 16 * s) * 4 : kNowhere);
      mark_steps = load_raw<float>(mark_sums.tile(chunk, p.seg > 0 && rows > 0), on ? cm * 4 : kNowhere);
    }
  };
  // what the tile's thread keeps of its row and channel from one chunk's staging to its outputs
  struct Row {
    float x, raw, z, dy, d, ds;
  };
  auto stage = [&](int buf, int chunk) {
    Row t;
    t.x = value_of<T>(xr), t.raw = value_of<T>(dr) + bias, t.z = value_of<T>(zr), t.dy = value_of<T>(gr);
    const float step = G.softplus ? softplus(t.raw) : t.raw;
    t.ds = GATE ? t.dy * t.z * row_sigmoid<T>(t.z) : t.dy;
    t.d = tile_on && chunk * kRows + r < p.len ? step : 0.f;   // (dy, and so ds, is zero there)
    s_d[buf][ch][r] = float2{t.d, t.d * t.x};
    s_ds[buf][ch][r] = t.ds;
    bc.stage(s_bc[buf]);
    return t;
  };
  Row row = {};
  if (p.ch0 < p.ch1) {
    fetch(p.ch1 - 1);
    row = stage(0, p.ch1 - 1);
    __syncthreads();
  }
  int buf = 0;
  for (int k = p.ch1 - 1; k >= p.ch0; --k, buf ^= 1) {
    const int row0 = k * kRows, rows = min(p.len - row0, kRows);
    float hc[NS];   // the state before the chunk
    if constexpr (MAIN) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        hc[s] = value_of<float>(mark[s]);
        if (p.seg > 0) hc[s] += Decay<EXACT>(value_of<float>(mark_steps) * A2[s]).of(start[s]);
      }
    }
    fetch(k - 1);
    float2 dd = s_d[buf][mine][n];
    const float dsm = s_ds[buf][mine][n];
    const float *Bl = s_bc[buf], *Cl = s_bc[buf] + (MAIN ? kRows * NS * 16 : 0);
    float Bv[kRows], Cv[kRows];   // of a block of rows
    if constexpr (!MAIN) {
      each<NS>([&](auto K) {
        constexpr int b = NS - 1 - K;
        load_block<NS, b>(Cv, Cl);
        each<kRows / NS>([&](auto J) {
          constexpr int i = kRows / NS - 1 - J, j = b * (kRows / NS) + i;
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const float R = __builtin_fmaf(row_bcast<j>(dsm), Cv[i * NS + s], Q[s]);
            Q[s] = Decay<EXACT>(row_bcast<j>(dd.x) * A2[s]).of(R);
          }
        });
      });
      stage(buf ^ 1, k - 1);
      lds_barrier();
    } else {
      Decay<EXACT> e[kRows][NS];
      float h[kRows][NS], sums[kRows];
      each<NS>([&](auto K) {
        constexpr int b = K;
        load_block<NS, b>(Bv, Bl);
        load_block<NS, b>(Cv, Cl);
        each<kRows / NS>([&](auto J) {
          constexpr int j = b * (kRows / NS) + J;
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            e[j][s] = Decay<EXACT>(row_bcast<j>(dd.x) * A2[s]);
            h[j][s] = e[j][s].of(j ? h[j ? j - 1 : 0][s] : hc[s], row_bcast<j>(dd.y) * Bv[J * NS + s]);
            if constexpr (GATE) sums[j] = s ? __builtin_fmaf(Cv[J * NS + s], h[j][s], sums[j]) : Cv[J * NS] * h[j][s];
          }
        });
      });
      if constexpr (GATE) s_out[buf][0][mine][n] = turn_sums(sums, n);
      // (so that the broadcasts below are operands of their products again, not values kept from above)
      pin_float(dd.x), pin_float(dd.y);
      float u[kRows], v[kRows], odd[NS];
      float* part = s_part[buf % kPartBufs][tid >> 6] + (tid & 63);
      each<NS>([&](auto K) {
        constexpr int b = NS - 1 - K;
        if constexpr (NS > 1) {   // (of one block they are still there)
          load_block<NS, b>(Bv, Bl);
          load_block<NS, b>(Cv, Cl);
        }
        each<kRows / NS>([&](auto J) {
          constexpr int i = kRows / NS - 1 - J, j = b * (kRows / NS) + i;
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const float R = __builtin_fmaf(row_bcast<j>(dsm), Cv[i * NS + s], Q[s]);
            // dC and dB of the wave's channels: in the halves of the wave, and two rows in their halves
            const float both = sum_halves(row_bcast<j>(dsm) * h[j][s], row_bcast<j>(dd.y) * R);
            if constexpr (j % 2) odd[s] = both;
            else part[(j / 2 * NS + s) * 64] = sum_quarters(both, odd[s]);
            u[j] = s ? __builtin_fmaf(R, Bv[i * NS + s], u[j]) : R * Bv[i * NS];
            Q[s] = e[j][s].of(R);
            const float q = Q[s] * (j ? h[j ? j - 1 : 0][s] : hc[s]);
            v[j] = s ? __builtin_fmaf(q, A[s], v[j]) : q * A[0];
            dA[s] = __builtin_fmaf(q, row_bcast<j>(dd.x), dA[s]);
          }
        });
      });
      s_out[buf][1][mine][n] = turn_sums(u, n);
      s_out[buf][2][mine][n] = turn_sums(v, n);
      const Row next = stage(buf ^ 1, k - 1);
      lds_barrier();
      {
        const float uu = s_out[buf][1][ch][r], dd_ = __builtin_fmaf(row.x, uu, s_out[buf][2][ch][r]);
        const float ddt = G.softplus ? dd_ * softplus_slope(row.raw) : dd_;
        store_elem<T>(dxs.tile(row0, rows), off, __builtin_fmaf(row.d, uu, Dc * row.ds));
        store_elem<T>(ddts.tile(row0, rows), off, ddt);
        if constexpr (GATE) {
          const float pre = __builtin_fmaf(Dc, row.x, s_out[buf][0][ch][r]);
          store_elem<T>(dzs.tile(row0, rows), off, row.dy * pre * silu_slope(row.z, row_sigmoid<T>(row.z)));
        }
        dD = __builtin_fmaf(row.ds, row.x, dD);
        dbias += r < rows ? ddt : 0.f;
      }
      // dC (lower half of a wave's lanes) and dB of the workgroup's channels; odd DPP rows hold the second of two rows
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int at = tid + i * kScanThreads, lane = at % 64, which = lane / 32;
        const int t = at / (64 * NS) * 2 + (lane / 16 & 1), m = lane % 16 + 16 * (at / 64 % NS);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += s_part[buf % kPartBufs][w][at];
        if (t < rows && m < G.N)
          L.w.bc[((((size_t)p.g * G.cblocks + p.cb) * G.B + p.b) * G.T + row0 + t) * 2 * G.N + which * G.N + m] = sum;
      }
      row = next;
      if constexpr (kPartBufs == 1) lds_barrier();   // the next chunk writes the same parts
    }
  }
  if constexpr (!MAIN) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (state[s]) L.w.back[((size_t)p.b * G.nseg + p.seg) * CN + (size_t)cm * G.N + n + 16 * s] = Q[s];
  } else {
    float* part = L.w.weights + ((size_t)p.b * G.nseg + p.seg) * (CN + 2 * (size_t)G.C);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (!state[s]) continue;
      part[(size_t)cm * G.N + n + 16 * s] = dA[s];
      if (p.seg == 0 && a.dh0) a.dh0[(size_t)p.b * CN + (size_t)cm * G.N + n + 16 * s] = Q[s];
    }
    // over the tile's rows: thread (r, ch) holds the sums of rows r, r + 16, ...
    __syncthreads();
    s_out[0][0][ch][r] = dD;
    s_out[0][1][ch][r] = dbias;
    __syncthreads();
    if (tid < 2 * kCh && c0 + tid % kCh < G.Cg) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) sum += s_out[0][tid / kCh][tid % kCh][i];
      part[CN + (size_t)(tid / kCh) * G.C + first_c + tid % kCh] = sum;
    }
    if (G.pad_zero && tile_on) {
      const T zero = from_f32<T>(0.f);
      const int to = min((p.ch0 + G.seg_chunks) * kRows, G.T);
      for (int t = max(p.len, p.ch0 * kRows) + r; t < to; t += kRows) {
        const size_t at = ((size_t)p.b * G.T + t) * G.C + ct;
        ((T*)a.dx)[at] = ((T*)a.ddt)[at] = zero;
        if (GATE) ((T*)a.dz)[at] = zero;
      }
    }
  }
}

// dBm and dCm: the sums of the channel blocks' parts
template <typename T> __global__ __launch_bounds__(256) void scan_bc_kernel(const ScanLaunch L) {
  const ScanGeom& G = L.G;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, GN = (long long)G.G * G.N;
  const long long row = i / (2 * GN);
  if (row >= (long long)G.B * G.T) return;
  const int rest = (int)(i - row * 2 * GN), which = rest / (int)GN, gn = rest - which * (int)GN;
  const int g = gn / G.N, m = gn - g * G.N, b = (int)(row / G.T), t = (int)(row - (long long)b * G.T);
  const int len = L.a.lens ? min(max(L.a.lens[b], 0), G.T) : G.T;
  T* out = (T*)(which ? L.a.dBm : L.a.dCm) + row * GN + gn;
  if (t >= len) {
    if (G.pad_zero) *out = from_f32<T>(0.f);
    return;
  }
  const size_t stride = (size_t)G.B * G.T * 2 * G.N;
  const float* part = L.w.bc + (size_t)g * G.cblocks * stride + ((size_t)row * 2 + which) * G.N + m;
  float sum = 0.f;
#pragma unroll 8
  for (int k = 0; k < G.cblocks; ++k) sum += part[k * stride];
  *out = from_f32<T>(sum);
}

// ---------------------------------------------------------------- decode

// Four states a lane, LPC lanes a channel (a power of two, up to 16), EACH
// sequences a thread, whose loads are in flight together (the weights are read
// once).  HBM-bound: the state is read and written once.
template <typename T, int LPC, bool WHOLE, int EACH>
__global__ __launch_bounds__(256) void scan_decode_kernel(const ScanLaunch L) {
  constexpr bool EXACT = sizeof(T) == 4;
  const SelScanArgs& a = L.a;
  const ScanGeom& G = L.G;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long group = i / LPC / G.C;   // of EACH sequences
  if (group * EACH >= G.B) return;         // (a channel's lanes all leave or all stay)
  const int l = (int)(i % LPC), n0 = 4 * l, left = G.N - n0;
  const int c = (int)(i / LPC - group * G.C), g = c / G.Cg;
  const float* ap = a.A + (size_t)c * G.N + n0;
  f32x4 A2 = zero4();
  if constexpr (WHOLE) {
    if (left > 0) A2 = *reinterpret_cast<const f32x4*>(ap);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) A2[e] = ap[e];
  }
  A2 *= kLog2e;
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, D = a.D ? a.D[c] : 0.f;
  RowVec<T, 4> Br[EACH], Cr[EACH];
  T xr[EACH], dr[EACH], zr[EACH];
  f32x4 h[EACH];
#pragma unroll
  for (int m = 0; m < EACH; ++m) {
    const long long b = group * EACH + m;
    const int some = b < G.B ? left : 0;
    const size_t channel = (size_t)(b < G.B ? b : group * EACH) * G.C + c, seq = channel / G.C;
    const float* hp = a.H_inout + channel * G.N + n0;
    const size_t bc = seq * G.ldbc + (size_t)g * G.N + n0;
    h[m] = zero4();
    if constexpr (WHOLE) {
      if (some > 0) h[m] = *reinterpret_cast<const f32x4*>(hp);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < some) h[m][e] = hp[e];
    }
    Br[m].load((const T*)a.Bm + bc, some);
    Cr[m].load((const T*)a.Cm + bc, some);
    xr[m] = ((const T*)a.x)[channel];
    dr[m] = ((const T*)a.dt)[channel];
    zr[m] = a.z ? ((const T*)a.z)[seq * G.ldz + c] : from_f32<T>(0.f);
  }
#pragma unroll
  for (int m = 0; m < EACH; ++m) {
    const long long b = group * EACH + m;
    if (b >= G.B) break;
    const size_t channel = (size_t)b * G.C + c;
    float* hp = a.H_inout + channel * G.N + n0;
    float Bv[4], Cv[4], s = 0.f;
    Br[m].widen(Bv);
    Cr[m].widen(Cv);
    const float x = to_f32(xr[m]);
    float d = to_f32(dr[m]) + bias;
    if (G.softplus) d = softplus(d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[m][e] = Decay<EXACT>(d * A2[e]).of(h[m][e], d * x * Bv[e]);
      s = __builtin_fmaf(Cv[e], h[m][e], s);
    }
    if constexpr (WHOLE) {
      if (left > 0) *reinterpret_cast<f32x4*>(hp) = h[m];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) hp[e] = h[m][e];
    }
    if constexpr (LPC > 1) s = group_sum<LPC>(s);
    if (l == 0) {
      float y = __builtin_fmaf(D, x, s);
      if (a.z) {
        const float z = to_f32(zr[m]);
        y *= z * row_sigmoid<T>(z);
      }
      ((T*)a.y)[channel] = from_f32<T>(y);
    }
  }
}

// ---------------------------------------------------------------- host

ScanGeom scan_geom(int B, int T, int C, int G, int N) {
  ScanGeom g = {};
  g.B = B, g.T = T, g.C = C, g.G = G, g.N = N;
  g.Cg = C / G;
  g.cblocks = (g.Cg + kCh - 1) / kCh;
  g.chunks = (int)(((long long)T + kRows - 1) / kRows);
  // Segments where the channels leave CUs without a workgroup; of 128 rows at least.
  const long long blocks = (long long)B * G * g.cblocks;
  g.nseg = 1;
  if (blocks > 0 && blocks < 192) g.nseg = (int)std::max(1LL, std::min((512 + blocks - 1) / blocks, (long long)g.chunks / 8));
  g.seg_chunks = std::max(1, (g.chunks + g.nseg - 1) / g.nseg);
  g.nseg = std::max(1, (g.chunks + g.seg_chunks - 1) / g.seg_chunks);
  return g;
}

struct ScanSizes {
  size_t ends, steps, back, marks, mark_steps, bc, weights;   // floats
};
ScanSizes scan_sizes(const ScanGeom& g, bool bwd) {
  auto up = [](size_t n) { return (n + 63) / 64 * 64; };
  const size_t CN = (size_t)g.C * g.N, segs = (size_t)g.B * g.nseg;
  ScanSizes s = {};
  if (g.nseg > 1) s.ends = up(segs * CN), s.steps = up(segs * g.C);
  if (!bwd) return s;
  if (g.nseg > 1) s.back = up(segs * CN), s.mark_steps = up((size_t)g.B * g.chunks * g.C);
  s.marks = up((size_t)g.B * g.chunks * CN);
  s.bc = up((size_t)g.G * g.cblocks * g.B * g.T * 2 * g.N);
  s.weights = up(segs * (CN + 2 * (size_t)g.C));
  return s;
}
size_t scan_bytes(const ScanSizes& s) {
  return 4 * (s.ends + s.steps + s.back + s.marks + s.mark_steps + s.bc + s.weights);
}

ScanLaunch scan_launch(const SelScanArgs& a, bool bwd) {
  ScanLaunch L;
  L.a = a;
  L.G = scan_geom(a.B, a.T, a.C, a.G, a.N);
  L.G.ldbc = a.ldbc, L.G.ldz = a.ldz, L.G.softplus = a.softplus, L.G.pad_zero = a.pad_zero;
  L.segs = L.G.nseg;
  const ScanSizes s = scan_sizes(L.G, bwd);
  float* p = (float*)a.workspace;
  auto take = [&](size_t n) { float* q = n ? p : nullptr; p = n ? p + n : p; return q; };
  L.w.ends = take(s.ends), L.w.steps = take(s.steps), L.w.back = take(s.back), L.w.marks = take(s.marks);
  L.w.mark_steps = take(s.mark_steps), L.w.bc = take(s.bc), L.w.weights = take(s.weights);
  return L;
}

unsigned scan_blocks(const ScanLaunch& L) {
  const int total = L.G.B * L.segs * L.G.G * L.G.cblocks;
  return (unsigned)((total + 7) / 8 * 8);
}

template <bool BACK> hipError_t launch_join(const ScanLaunch& L) {
  const unsigned blocks = (unsigned)(((long long)L.G.B * L.G.C * L.G.N + 255) / 256);
  if (L.a.dtype == CKDA_DTYPE_F32) hipLaunchKernelGGL((scan_join_kernel<true, BACK>), dim3(blocks), dim3(256), 0, L.a.stream, L);
  else hipLaunchKernelGGL((scan_join_kernel<false, BACK>), dim3(blocks), dim3(256), 0, L.a.stream, L);
  return hipGetLastError();
}

// Channels of the forward's workgroups: 16 rather than the backward's 32 (which share one part of dB and dC), for
// barriers among fewer waves (MI355X, us, 16 and 32 channels: B4 T4096 C2048 N16 233 and 243, B16 T1024 C4096 339
// and 357, B2 T2048 C2048 N64 221 and 270; 8 channels are slower again, 237, 367 and 261).
constexpr int kFwdCh = 16;
template <typename T, int NS> hipError_t launch_fwd_t(const SelScanArgs& a) {
  ScanLaunch L = scan_launch(a, false);
  L.G.cblocks = (L.G.Cg + kFwdCh - 1) / kFwdCh;
  if (L.G.nseg > 1) {
    L.segs = L.G.nseg - 1;
    hipLaunchKernelGGL((scan_fwd_kernel<T, NS, kFwdCh, false, false, true>), dim3(scan_blocks(L)), dim3(kRows * kFwdCh), 0, a.stream, L);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = launch_join<false>(L);
    if (e != hipSuccess) return e;
    L.segs = L.G.nseg;
  }
  hipLaunchKernelGGL((scan_fwd_kernel<T, NS, kFwdCh, true, false, false>), dim3(scan_blocks(L)), dim3(kRows * kFwdCh), 0, a.stream, L);
  return hipGetLastError();
}

template <typename T, int NS, bool MAIN> void launch_bwd_kernel(const ScanLaunch& L) {
  if (L.a.z)
    hipLaunchKernelGGL((scan_bwd_kernel<T, NS, MAIN, true>), dim3(scan_blocks(L)), dim3(kScanThreads), 0, L.a.stream, L);
  else
    hipLaunchKernelGGL((scan_bwd_kernel<T, NS, MAIN, false>), dim3(scan_blocks(L)), dim3(kScanThreads), 0, L.a.stream, L);
}

template <typename T, int NS> hipError_t launch_bwd_t(const SelScanArgs& a) {
  ScanLaunch L = scan_launch(a, true);
  hipError_t e = hipSuccess;
  if (L.G.B > 0) {
    if (L.G.nseg > 1)
      hipLaunchKernelGGL((scan_fwd_kernel<T, NS, kCh, false, true, true>), dim3(scan_blocks(L)), dim3(kScanThreads), 0, a.stream, L);
    else
      hipLaunchKernelGGL((scan_fwd_kernel<T, NS, kCh, false, true, false>), dim3(scan_blocks(L)), dim3(kScanThreads), 0, a.stream, L);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (L.G.nseg > 1) {
      if ((e = launch_join<false>(L)) != hipSuccess) return e;
      L.segs = L.G.nseg - 1;
      launch_bwd_kernel<T, NS, false>(L);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      if ((e = launch_join<true>(L)) != hipSuccess) return e;
      L.segs = L.G.nseg;
    }
    launch_bwd_kernel<T, NS, true>(L);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const long long each = (long long)a.B * a.T * 2 * a.G * a.N;
    if (each > 0) {
      hipLaunchKernelGGL((scan_bc_kernel<T>), dim3((unsigned)((each + 255) / 256)), dim3(256), 0, a.stream, L);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  const size_t CN = (size_t)a.C * a.N, C = (size_t)a.C;
  return launch_part_sums(PartSums{L.w.weights, L.G.B * L.G.nseg, CN + 2 * C, {a.dA, a.dD, a.dbias}, {CN, C, C}}, a.stream);
}

// Two sequences a thread where that leaves threads enough (MI355X, us, one and two: 256 sequences of 4096 channels
// with 16 states 32.5 and 28, 64 of 2048 with 64 states 19.1 and 17).
template <typename T, int LPC, bool WHOLE> hipError_t launch_decode_t(const SelScanArgs& a) {
  const ScanLaunch L = scan_launch(a, false);
  const bool many = (long long)a.B * a.C * LPC >= 1 << 20;
  const long long groups = many ? (a.B + 1) / 2 : a.B;
  const unsigned blocks = (unsigned)((groups * a.C * LPC + 255) / 256);
  if (many) hipLaunchKernelGGL((scan_decode_kernel<T, LPC, WHOLE, 2>), dim3(blocks), dim3(256), 0, a.stream, L);
  else hipLaunchKernelGGL((scan_decode_kernel<T, LPC, WHOLE, 1>), dim3(blocks), dim3(256), 0, a.stream, L);
  return hipGetLastError();
}

template <typename T> hipError_t launch_scan(const SelScanArgs& a, bool bwd) {
  if (a.N <= 16) return bwd ? launch_bwd_t<T, 1>(a) : launch_fwd_t<T, 1>(a);
  if (a.N <= 32) return bwd ? launch_bwd_t<T, 2>(a) : launch_fwd_t<T, 2>(a);
  return bwd ? launch_bwd_t<T, 4>(a) : launch_fwd_t<T, 4>(a);
}

template <typename T, bool WHOLE> hipError_t launch_decode_n(const SelScanArgs& a) {
  if (a.N <= 4) return launch_decode_t<T, 1, WHOLE>(a);
  if (a.N <= 8) return launch_decode_t<T, 2, WHOLE>(a);
  if (a.N <= 16) return launch_decode_t<T, 4, WHOLE>(a);
  if (a.N <= 32) return launch_decode_t<T, 8, WHOLE>(a);
  return launch_decode_t<T, 16, WHOLE>(a);
}
template <typename T> hipError_t launch_decode(const SelScanArgs& a) {
  return a.N % 4 == 0 ? launch_decode_n<T, true>(a) : launch_decode_n<T, false>(a);
}

}  // namespace

size_t scan_fwd_workspace_bytes(int B, int T, int C, int G, int N) {
  return scan_bytes(scan_sizes(scan_geom(B, T, C, G, N), false));
}
size_t scan_bwd_workspace_bytes(int B, int T, int C, int G, int N) {
  return scan_bytes(scan_sizes(scan_geom(B, T, C, G, N), true));
}

// fewer than 2^32 threads in every launch, and counts of workgroups in an int
bool scan_fits_grid(int B, int T, int C, int G, int N) {
  const ScanGeom g = scan_geom(B, T, C, G, N);
  const long long blocks = (long long)B * g.nseg * G * g.cblocks;
  return blocks < (1LL << 22) && (long long)B * C * N < (1LL << 31) && (long long)B * C * 16 < (1LL << 31) &&
         (double)B * T * 2 * G * N < 4e9;
}

hipError_t launch_scan_fwd(const SelScanArgs& a) {
  return a.dtype == CKDA_DTYPE_BF16 ? launch_scan<bf16_t>(a, false) : launch_scan<float>(a, false);
}
hipError_t launch_scan_bwd(const SelScanArgs& a) {
  return a.dtype == CKDA_DTYPE_BF16 ? launch_scan<bf16_t>(a, true) : launch_scan<float>(a, true);
}
hipError_t launch_scan_decode(const SelScanArgs& a) {
  return a.dtype == CKDA_DTYPE_BF16 ? launch_decode<bf16_t>(a) : launch_decode<float>(a);
}

}  // namespace ckda
