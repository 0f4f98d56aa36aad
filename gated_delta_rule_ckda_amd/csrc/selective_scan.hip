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
// exponential and two fused products, and whatever else runs for each.  MI355X, B4 T4096
// C2048 N16 bf16 with the gate: forward 213 us (9.7 instructions for each state of a row,
// the vector units busy 72% of the time at the two waves a SIMD gets from 8192 channels),
// backward 632 (a pass forward 175, 10 instructions, and the main pass 435, 27; both with
// the vector units busy all the time).  fp32 367 and 983: its decays branch (see Decay).  Eight issue slots of 16 lanes for a state
// (the exponential takes four) would be 109 us, HBM 55.  The layout leaves little else to
// do for each:
//  * LN neighbouring lanes are one channel, each with NS states in registers, time
//    down a loop.  4 x 4 for up to 16 states; 16 x 2 and 16 x 4 for up to 32 and 64;
//    16 x 1 where 4 lanes a channel would leave SIMDs idle and the sequence would
//    have to be cut (see scan_plan).
//  * Rows go by chunks of 16.  What a row has for each channel (d, d x, ds) is made
//    once, by one lane, and handed to the channel's lanes by a DPP broadcast inside a
//    row of 16 lanes or a quad.
//  * Sums over the states (s, u, v) are made for LN rows at once by a transposing
//    reduction, which leaves each row's sum in a lane of its own (16 sums of 16
//    lanes: 33 instructions instead of 64), and what follows is again done once for
//    each row and channel.
//  * Sums over the channels (dB, dC) go the same way: values of different states and
//    rows are paired, each half of the lanes keeps one of the two.  The waves' sums
//    meet in LDS.  (On the fp32 matrix cores, 16x16x4, each masked row's product
//    takes 32 cycles in which the SIMD issues nothing else: slower, 1058 us against
//    830 at B4 T4096 C2048 N16.)
//  * Workgroups share B_t and C_t in LDS, as fp32; rows of x, dt, z, dy and y are
//    read and written by whole rows of the workgroup's channels and turned in LDS.
// Few channels and many rows: the sequence runs in segments.  A first pass makes
// each segment's own end state, a second joins them (a segment's decay is exp(A
// sum d), closed), the main pass starts from the joined states.  The backward needs
// the states in reverse: a pass forward in time stores them every 16 rows (8 with 4
// lanes; of its segment, joined when read), and the main pass recomputes the others in registers.  The
// segments' own gradient states, sum_t (a_1 .. a_t) ds_t C_t, take no second
// exponential: the same pass sums them with the running product of its decays.
#include <limits.h>

#include <algorithm>
#include <utility>

#include "ckda_internal.hpp"
#include "part_sums.hpp"
#include "row_vec.hpp"

namespace ckda {

namespace {

constexpr int kRows = 16;       // rows of a chunk
constexpr int kPad = kRows + 1;   // row of a turned tile in LDS
// Registers: for four waves on a SIMD with 4 lanes a channel, for two to four with 16 (rows' operands are loaded
// ahead, not one after the other); the backward's main pass with 4 lanes for three, which bf16 has without spills (fp32
// keeps 21 registers in memory with the gate and 6 without; with 16 lanes of four states 54 and 48).
#define CKDA_SCAN_WAVES(LN) __attribute__((amdgpu_waves_per_eu((LN) == 4 ? 4 : 2, 4)))
#define CKDA_SCAN_BWD_WAVES(LN) __attribute__((amdgpu_waves_per_eu((LN) == 4 ? 3 : 2, 4)))
constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = 1.9259629911266174e-8f, kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- lanes

template <int... J, typename F> __device__ __forceinline__ void each_impl(std::integer_sequence<int, J...>, F&& f) {
  (f(std::integral_constant<int, J>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F&& f) {
  each_impl(std::make_integer_sequence<int, N>{}, f);
}

// LN lanes a channel with NS states each
template <int LN, int NS> struct Layout {
  static constexpr int kStates = LN * NS;       // of a channel, the last ones possibly none
  static constexpr int kRegs = kRows / LN;      // registers that hold one value for each row of a chunk: row i LN + l in lane l of i
  static constexpr int kPack = 4 / NS;          // rows of B or C in one 16-byte LDS read
  static constexpr int kBlockRows = NS == 4 ? 1 : kRows / NS;   // rows whose B and C are read together,
  static constexpr int kBlock = kBlockRows * NS;                // and the values of a lane in them
  static constexpr int kBlocks = kRows / kBlockRows;            // of a chunk
  static constexpr int kMarks = LN == 4 ? 2 : 1;                // states of a chunk that the backward's first pass leaves
};

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
// (The compiler does not see what the asm reads and writes by vector instructions: the two wait states that a DPP
// source needs behind its writer stand at its start, and where a result goes to a DPP operand or a lane swap, two
// stand at its end.  Of turn_sums none does: the selects read them.)
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
// Values that the next chunk takes over are pinned where they are made: the compiler would move the arithmetic
// behind the branches that follow, and keep every operand until then.
template <int N> __device__ __forceinline__ void pin_floats(float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) pin_float(x[i]);
}

// The channel's value of row J, in all of its lanes.  Used by one state it is the DPP operand of its product; by
// several, a register of its own (kept apart from the products: each with a DPP operand would cost more).
template <int LN, int NS, int J> __device__ __forceinline__ float row_value(const float (&x)[kRows / LN]) {
  float v;
  if constexpr (LN == 16) v = row_bcast<J>(x[0]);
  else v = dpp_mov<(J % 4) * 0x55>(x[J / 4]);   // quad_perm [j,j,j,j]
  if constexpr (NS > 1) pin_float(v);
  return v;
}

// Sums over a channel's lanes of LN values, value j's sum to lane j
__device__ __forceinline__ float turn_quad(const float (&v)[4], int lane) {
  const bool two = lane & 2, one = lane & 1;
  const float c0 = (two ? v[2] : v[0]) + dpp_mov<0x4E>(two ? v[0] : v[2]);
  const float c1 = (two ? v[3] : v[1]) + dpp_mov<0x4E>(two ? v[1] : v[3]);
  return (one ? c1 : c0) + dpp_mov<0xB1>(one ? c0 : c1);
}
template <int LN> __device__ __forceinline__ float turn_lanes(const float (&v)[LN], int l) {
  if constexpr (LN == 16) return turn_sums(v, l);
  else return turn_quad(v, l);
}

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

// Sums over the 4 quads of a DPP row of 4 states of two quantities: quad b gets the sum of state (b & 1) 2 + b / 2
// of each.  Pairs across quads two apart (row_ror:8), then next ones (from the quad behind, row_ror:12, where the
// first of a pair is kept, from the one before, row_ror:4, where the second is).  The lane swap of sum_halves reads
// the results: its two wait states are the last instruction.
#define CKDA_QUADS(d, a, b, low, high, mask)                               \
  "v_add_f32_dpp " d ", " a ", " a " " low " row_mask:0xf bank_mask:0xf\n" \
  "v_add_f32_dpp " d ", " b ", " b " " high " row_mask:0xf bank_mask:" mask "\n"
__device__ __forceinline__ void sum_quads(const float (&x)[4], const float (&y)[4], float& sx, float& sy) {
  float a0, a1, a2, a3;
  asm("s_nop 1\n"   //
      CKDA_QUADS("%2", "%6", "%7", "row_ror:8", "row_ror:8", "0xc") CKDA_QUADS("%3", "%8", "%9", "row_ror:8", "row_ror:8", "0xc")
      CKDA_QUADS("%4", "%10", "%11", "row_ror:8", "row_ror:8", "0xc") CKDA_QUADS("%5", "%12", "%13", "row_ror:8", "row_ror:8", "0xc")
      CKDA_QUADS("%0", "%2", "%3", "row_ror:12", "row_ror:4", "0xa") CKDA_QUADS("%1", "%4", "%5", "row_ror:12", "row_ror:4", "0xa")
      "s_nop 1"
      : "=&v"(sx), "=&v"(sy), "=&v"(a0), "=&v"(a1), "=&v"(a2), "=&v"(a3)
      : "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "v"(y[0]), "v"(y[1]), "v"(y[2]), "v"(y[3]));
}
#undef CKDA_QUADS

// ---------------------------------------------------------------- elements

// exp(-|v|): with fp32 inputs to a few 2^-24 (the product with log2 e in two parts),
// with bf16 ones to (|v| + 2) 2^-24.
template <bool EXACT> __device__ __forceinline__ float exp_neg_abs(float v) {
  if constexpr (!EXACT) return __builtin_amdgcn_exp2f(fabsf(v) * -kLog2e);
  const float m = fminf(fabsf(v), 200.f), t = -m * kLog2e;
  const float lo = __builtin_fmaf(-m, kLog2eLo, __builtin_fmaf(-m, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, lo * kLn2, e);
}
// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|), with log((1 + r) / (1 - r)) =
// 2 r (1 + z f(z)), r = e / (2 + e) <= 1/3, z = r^2: small steps keep their relative
// accuracy, which log(1 + e) does not.  f is a polynomial fitted to least largest error
// over z <= 1/9: 2^-27 of the whole for fp32 inputs, 2^-22 for bf16.
template <bool EXACT> __device__ __forceinline__ float softplus(float v) {
  const float e = exp_neg_abs<EXACT>(v), r = e * __builtin_amdgcn_rcpf(2.f + e), z = r * r;
  float p, most;
  if constexpr (EXACT) {
    p = __builtin_fmaf(0.14005993f, z, 0.14000903f);
    p = __builtin_fmaf(p, z, 0.20010763f);
    p = __builtin_fmaf(p, z, 0.33333209f);
    most = v < 0.f ? 0.f : v;   // (a NaN stays one)
  } else {
    p = __builtin_fmaf(0.16991776f, z, 0.19817986f);
    p = __builtin_fmaf(p, z, 0.33336741f);
    most = fmaxf(v, 0.f);       // (a NaN stays one in e)
  }
  return __builtin_fmaf(2.f, __builtin_fmaf(r * z, p, r), most);
}
template <bool EXACT> __device__ __forceinline__ float softplus_slope(float v) {
  const float e = exp_neg_abs<EXACT>(v), r = __builtin_amdgcn_rcpf(1.f + e);
  return v >= 0.f ? r : e * r;
}

// A decay 2^x.  Where the inputs are bf16: itself, by the hardware's exponential
// (mean error -0.12 of 2^-24 for small x, so a state that remembers M rows is off
// by some 7e-9 M).  Where they are fp32: for -x < 1/16 its distance from 1, which
// keeps slow decays to 2^-24 of their rate (degree 4: next term 2^-25); stronger
// ones, of states that remember fewer than 24 rows, themselves.  The choice becomes
// branches, not selects: 147 regions under a mask in the 4-lane forward where bf16 has
// 20; both sides run where a wave's lanes differ, and nothing moves across them.
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

struct ScanWork {            // workspace of a call; P = a layout's states
  float* ends;               // [B][nseg][C][P]: segments' own end states, then start states
  float* steps;              // [B][nseg][C]: sums of d over the segments
  float* back;               // [B][nseg][C][P]: backward in time
  float* marks;              // [B][chunks kMarks][C][P]: states before each chunk (and in its middle), of their segment
  float* mark_steps;         // [B][chunks kMarks][C]: sums of d from the segment's start to each of those (nseg > 1)
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
// states of a lane, next to each other
template <int NS> __device__ __forceinline__ void load_states(uint32_t (&v)[NS], __amdgpu_buffer_rsrc_t r, int off) {
  if constexpr (NS == 4) {
    const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
    v[0] = w[0], v[1] = w[1], v[2] = w[2], v[3] = w[3];
  } else if constexpr (NS == 2) {
    const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
    v[0] = w[0], v[1] = w[1];
  } else {
    v[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  }
}
template <int NS> __device__ __forceinline__ void store_states(__amdgpu_buffer_rsrc_t r, int off, const float (&h)[NS]) {
  if constexpr (NS == 4)
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(h[0]), __float_as_uint(h[1]), __float_as_uint(h[2]), __float_as_uint(h[3])}, r, off, 0, 0);
  else if constexpr (NS == 2)
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(h[0]), __float_as_uint(h[1])}, r, off, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(h[0]), r, off, 0, 0);
}
// A prefetched element, widened here and not where it was loaded (which would wait for it there).
template <typename T> __device__ __forceinline__ float value_of(uint32_t raw) {
  pin(raw);
  return __uint_as_float(sizeof(T) == 2 ? raw << 16 : raw);
}

// B and C (either alone: WHICH 1 or 2, both: 3) of SUBS chunks of rows in LDS, each
// as [row / kPack][lane][row % kPack][state], 16 bytes a lane.  Every wave moves one of
// the two at a time.
template <typename T, int LN, int NS, int SUBS, int THREADS, int WHICH> struct BcTile {
  using Lay = Layout<LN, NS>;
  static constexpr int kOne = SUBS * kRows * Lay::kStates;             // elements of one of the two
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
      const int idx = place_of(i), n = idx % Lay::kStates;
      off[i] = n < L.G.N && !idle() ? (idx / Lay::kStates * L.G.ldbc + p.g * L.G.N + n) * (int)sizeof(T) : kNowhere;
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
      const int idx = place_of(i), n = idx % Lay::kStates, row = idx / Lay::kStates;
      const int at = (row / Lay::kPack * LN + n / NS) * 4 + row % Lay::kPack * NS + n % NS;
      if (!idle()) s[(of_c(i) && WHICH == 3 ? kOne : 0) + at] = value_of<T>(raw[i]);
    }
  }
};

// Block K of a tile's B or C: f[row * NS + s] of this lane's states.
template <int LN, int NS, int K, int VALUES> __device__ __forceinline__ void load_block(float (&f)[VALUES], const float* one) {
  static_assert(VALUES == Layout<LN, NS>::kBlock, "values of a block");
  constexpr int Q = VALUES / 4;
  const f32x4* p = reinterpret_cast<const f32x4*>(one) + K * Q * LN + threadIdx.x % LN;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const f32x4 v = p[q * LN];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * q + i] = v[i];
  }
}

// ---------------------------------------------------------------- forward

// MAIN: outputs (and the last state) from the segments' start states.  Else: the
// segments' own end states and sums of steps.  SUBS chunks of rows between barriers.
template <typename T, int LN, int NS, int THREADS, int SUBS, bool MAIN>
__global__ __launch_bounds__(THREADS) CKDA_SCAN_WAVES(LN) void scan_fwd_kernel(const ScanLaunch L) {
  using Lay = Layout<LN, NS>;
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int CH = THREADS / LN, REGS = Lay::kRegs, TILE = SUBS * kRows, EACH = SUBS * REGS, P = Lay::kStates;
  __shared__ float2 s_d[2][SUBS][CH][kPad];
  __shared__ float s_y[MAIN ? 2 : 1][MAIN ? SUBS : 1][MAIN ? CH : 1][kPad];
  __shared__ __attribute__((aligned(16))) float s_bc[2][TILE * P * (MAIN ? 2 : 1)];
  const SelScanArgs& a = L.a;
  const ScanGeom& G = L.G;
  ScanPlace p;
  if (!scan_place(L, p)) return;
  const int tid = threadIdx.x, l = tid % LN, mine = tid / LN;   // lane and channel in the recurrence
  const int r = tid / CH, ch = tid % CH;                         // row (i LN + r) and channel of the tiles
  const int c0 = p.cb * CH, first_c = p.g * G.Cg + c0;
  const bool on = c0 + mine < G.Cg, tile_on = c0 + ch < G.Cg;
  const int cm = first_c + mine, ct = first_c + ch;
  const int row0 = p.ch0 * kRows, end = min(p.ch1 * kRows, p.len);   // rows of the segment

  float A2[NS], h[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int n = l * NS + s;
    const bool state = on && n < G.N;
    A2[s] = state ? a.A[(size_t)cm * G.N + n] * kLog2e : 0.f;
    h[s] = 0.f;
    if (state) {
      // (of several segments the first one's start too: its h0 may be the hT that the last one writes)
      if (MAIN && G.nseg > 1) h[s] = L.w.ends[(((size_t)p.b * G.nseg + p.seg) * G.C + cm) * P + n];
      else if (p.seg == 0 && a.h0) h[s] = a.h0[((size_t)p.b * G.C + cm) * G.N + n];
    }
  }
  const float bias = tile_on && a.dt_bias ? a.dt_bias[ct] : 0.f;
  const float Dc = MAIN && tile_on && a.D ? a.D[ct] : 0.f;

  const size_t first = (size_t)p.b * G.T + row0;
  const Rows<T> xs(a.x, first, G.C), ds(a.dt, first, G.C), ys(a.y, first, G.C), zs(a.z, first, G.ldz);
  const Rows<T> Bs(a.Bm, first, G.ldbc), Cs(a.Cm, first, G.ldbc);
  int off[EACH], zoff[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    off[i] = tile_on ? ((i * LN + r) * G.C + ct) * (int)sizeof(T) : kNowhere;
    zoff[i] = tile_on ? ((i * LN + r) * G.ldz + ct) * (int)sizeof(T) : kNowhere;
  }
  uint32_t xr[EACH], dr[EACH], zr[EACH] = {};
  BcTile<T, LN, NS, SUBS, THREADS, MAIN ? 3 : 1> bc;
  bc.place(L, p);
  // Rows behind the segment read zero; no branch around the loads (values that meet behind one are copied there,
  // and the copies wait for the loads).
  auto fetch = [&](int t0) {
    const int rows = min(end - t0, TILE), row = t0 - row0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      xr[i] = load_raw<T>(xs.tile(row, rows), off[i]);
      dr[i] = load_raw<T>(ds.tile(row, rows), off[i]);
      if (MAIN) zr[i] = load_raw<T>(zs.tile(row, a.z ? rows : 0), zoff[i]);
    }
    bc.fetch(Bs, Cs, row, rows);
  };
  auto stage = [&](int buf, int t0) {
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      float d = value_of<T>(dr[i]) + bias;
      if (G.softplus) d = softplus<EXACT>(d);
      d = tile_on && t0 + i * LN + r < end ? d : 0.f;   // a step of zero leaves the state
      s_d[buf][i / REGS][ch][i % REGS * LN + r] = float2{d, d * value_of<T>(xr[i])};
    }
    bc.stage(s_bc[buf]);
  };

  float steps = 0.f;
  if (row0 < end) {
    fetch(row0);
    stage(0, row0);
    __syncthreads();
  }
  int buf = 0;
  for (int t0 = row0; t0 < end; t0 += TILE, buf ^= 1) {
    uint32_t xk[EACH], zk[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) xk[i] = xr[i], zk[i] = zr[i];
    const bool more = t0 + TILE < end;
    fetch(t0 + TILE);
    // B and C of a block of rows are loaded while the block before is worked on
    const float* one = s_bc[buf];
    float d[SUBS][REGS], dx[SUBS][REGS], Bv[2][Lay::kBlock], Cv[2][Lay::kBlock];
    load_block<LN, NS, 0>(Bv[0], one);
    if constexpr (MAIN) load_block<LN, NS, 0>(Cv[0], one + TILE * P);
#pragma unroll
    for (int i = 0; i < SUBS; ++i)
#pragma unroll
      for (int q = 0; q < REGS; ++q) {
        const float2 v = s_d[buf][i][mine][q * LN + l];
        d[i][q] = v.x, dx[i][q] = v.y;
      }
    float sums[LN];
    each<SUBS * Lay::kBlocks>([&](auto K) {
      constexpr int k = K, i = k / Lay::kBlocks, b = k % Lay::kBlocks, R = Lay::kBlockRows;   // a block, its chunk and its place there
      if constexpr (k + 1 < SUBS * Lay::kBlocks) {
        load_block<LN, NS, k + 1>(Bv[(k + 1) % 2], one);
        if constexpr (MAIN) load_block<LN, NS, k + 1>(Cv[(k + 1) % 2], one + TILE * P);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (!MAIN && b == 0) {
        float sum = d[i][0];
#pragma unroll
        for (int q = 1; q < REGS; ++q) sum += d[i][q];
        steps += group_sum<LN>(sum);
      }
      each<R>([&](auto J) {
        constexpr int j = b * R + J;
        const float dj = row_value<LN, NS, j>(d[i]), dxj = row_value<LN, NS, j>(dx[i]);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          h[s] = Decay<EXACT>(dj * A2[s]).of(h[s], dxj * Bv[k % 2][J * NS + s]);
          if constexpr (MAIN) sums[j % LN] = s ? __builtin_fmaf(Cv[k % 2][J * NS + s], h[s], sums[j % LN]) : Cv[k % 2][J * NS] * h[s];
        }
      });
      pin_floats(h);
      if constexpr (MAIN && (b + 1) * R % LN == 0) s_y[buf][i][mine][(b + 1) * R - LN + l] = turn_lanes<LN>(sums, l);
    });
    if (more) stage(buf ^ 1, t0 + TILE);
    lds_barrier();
    if constexpr (MAIN) {
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        float y = __builtin_fmaf(Dc, value_of<T>(xk[i]), s_y[buf][i / REGS][ch][i % REGS * LN + r]);
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
        if (l * NS + s < G.N) a.hT[((size_t)p.b * G.C + cm) * G.N + l * NS + s] = h[s];
    }
    if (G.pad_zero && tile_on) {
      const int to = (int)min(((long long)p.ch0 + G.seg_chunks) * kRows, (long long)G.T);
      for (int t = max(p.len, row0) + r; t < to; t += LN) ((T*)a.y)[((size_t)p.b * G.T + t) * G.C + ct] = from_f32<T>(0.f);
    }
  } else if (on) {
#pragma unroll
    for (int s = 0; s < NS; ++s) L.w.ends[(((size_t)p.b * G.nseg + p.seg) * G.C + cm) * P + l * NS + s] = h[s];
    if (l == 0) L.w.steps[((size_t)p.b * G.nseg + p.seg) * G.C + cm] = steps;
  }
}

// Segments' own states joined in order, in place: each place gets the state that its
// segment starts from.  Backward in time the gradients of their last states, from dhT
// on, by the second half of the workgroups (one launch: 5 us less than two).
template <bool EXACT> __global__ __launch_bounds__(256) void scan_join_kernel(const ScanLaunch L, int P, unsigned half) {
  const ScanGeom& G = L.G;
  const bool back = blockIdx.x >= half;
  const long long i = (long long)(blockIdx.x - (back ? half : 0)) * 256 + threadIdx.x, CP = (long long)G.C * P;
  if (i >= (long long)G.B * CP) return;
  const int b = (int)(i / CP), c = (int)(i % CP / P), n = (int)(i % P);
  if (n >= G.N) return;
  const float A2 = L.a.A[(size_t)c * G.N + n] * kLog2e;
  float* own = (back ? L.w.back : L.w.ends) + (size_t)b * G.nseg * CP + i % CP;
  const float* steps = L.w.steps + (size_t)b * G.nseg * G.C + c;
  const float* first = back ? L.a.dhT : L.a.h0;
  float h = first ? first[((size_t)b * G.C + c) * G.N + n] : 0.f;
  constexpr int EACH = 8;   // segments whose loads are in flight together (64 segments: 20 us one after the other, 8 so)
  for (int k0 = 0; k0 < G.nseg; k0 += EACH) {
    float next[EACH], sum[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      // (of the last one nobody needs the end, and the forward does not make it)
      const int k = min(k0 + i, G.nseg - 2), seg = back ? G.nseg - 1 - k : k;
      next[i] = own[(size_t)seg * CP], sum[i] = steps[(size_t)seg * G.C];
    }
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int k = k0 + i;
      if (k >= G.nseg) break;
      own[(size_t)(back ? G.nseg - 1 - k : k) * CP] = h;
      // (the first segment's own state has the initial one in it already)
      h = back || k ? Decay<EXACT>(sum[i] * A2).of(h) + next[i] : next[i];
    }
  }
}

// ---------------------------------------------------------------- backward

// What the main pass needs from a pass forward in time: the states before each chunk
// (with 4 lanes also in its middle: the main pass has registers for the states of 8 rows) and, of several segments (SEGS), each segment's own end state, its sum of steps, and
// its own gradient state (of the state before it, from its rows alone).
template <typename T, int LN, int NS, int THREADS, bool SEGS>
__global__ __launch_bounds__(THREADS) CKDA_SCAN_WAVES(LN) void scan_prep_kernel(const ScanLaunch L) {
  using Lay = Layout<LN, NS>;
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr int CH = THREADS / LN, REGS = Lay::kRegs, P = Lay::kStates;
  __shared__ float2 s_d[2][CH][kPad];
  __shared__ float s_ds[SEGS ? 2 : 1][SEGS ? CH : 1][kPad];
  __shared__ __attribute__((aligned(16))) float s_bc[2][kRows * P * (SEGS ? 2 : 1)];
  const SelScanArgs& a = L.a;
  const ScanGeom& G = L.G;
  ScanPlace p;
  if (!scan_place(L, p)) return;
  const int tid = threadIdx.x, l = tid % LN, mine = tid / LN;
  const int r = tid / CH, ch = tid % CH;
  const int c0 = p.cb * CH, first_c = p.g * G.Cg + c0;
  const bool on = c0 + mine < G.Cg, tile_on = c0 + ch < G.Cg;
  const int cm = first_c + mine, ct = first_c + ch;

  float A2[NS], h[NS], Q[NS], product[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int n = l * NS + s;
    const bool state = on && n < G.N;
    A2[s] = state ? a.A[(size_t)cm * G.N + n] * kLog2e : 0.f;
    h[s] = state && p.seg == 0 && a.h0 ? a.h0[((size_t)p.b * G.C + cm) * G.N + n] : 0.f;
    Q[s] = 0.f, product[s] = 1.f;
  }
  const float bias = tile_on && a.dt_bias ? a.dt_bias[ct] : 0.f;
  const size_t first = (size_t)p.b * G.T;
  const Rows<T> xs(a.x, first, G.C), dts(a.dt, first, G.C), dys(a.dy, first, G.C), zs(a.z, first, G.ldz);
  const Rows<T> Bs(a.Bm, first, G.ldbc), Cs(a.Cm, first, G.ldbc);
  constexpr int MARKS = Lay::kMarks;
  const size_t first_mark = (size_t)p.b * G.chunks * MARKS;
  const Rows<float> marks(L.w.marks, first_mark, G.C * P), mark_sums(L.w.mark_steps, first_mark, G.C);
  const int moff = on ? (cm * P + l * NS) * 4 : kNowhere;
  int off[REGS], zoff[REGS];
#pragma unroll
  for (int i = 0; i < REGS; ++i) {
    off[i] = tile_on ? ((i * LN + r) * G.C + ct) * (int)sizeof(T) : kNowhere;
    zoff[i] = tile_on ? ((i * LN + r) * G.ldz + ct) * (int)sizeof(T) : kNowhere;
  }
  uint32_t xr[REGS], dr[REGS], gr[REGS] = {}, zr[REGS] = {};
  BcTile<T, LN, NS, 1, THREADS, SEGS ? 3 : 1> bc;
  bc.place(L, p);
  auto fetch = [&](int chunk) {
    const int row = chunk * kRows, rows = chunk < p.ch1 ? min(p.len - row, kRows) : 0;
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      xr[i] = load_raw<T>(xs.tile(row, rows), off[i]);
      dr[i] = load_raw<T>(dts.tile(row, rows), off[i]);
      if (SEGS) {
        gr[i] = load_raw<T>(dys.tile(row, rows), off[i]);
        zr[i] = load_raw<T>(zs.tile(row, a.z ? rows : 0), zoff[i]);
      }
    }
    bc.fetch(Bs, Cs, row, rows);
  };
  auto stage = [&](int buf, int chunk) {
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      float d = value_of<T>(dr[i]) + bias;
      if (G.softplus) d = softplus<EXACT>(d);
      d = tile_on && chunk * kRows + i * LN + r < p.len ? d : 0.f;
      s_d[buf][ch][i * LN + r] = float2{d, d * value_of<T>(xr[i])};
      if constexpr (SEGS) {
        const float z = value_of<T>(zr[i]);
        s_ds[buf][ch][i * LN + r] = value_of<T>(gr[i]) * (a.z ? z * row_sigmoid<T>(z) : 1.f);   // (dy is zero behind the rows)
      }
    }
    bc.stage(s_bc[buf]);
  };
  float steps = 0.f;
  if (p.ch0 < p.ch1) {
    fetch(p.ch0);
    stage(0, p.ch0);
    __syncthreads();
  }
  int buf = 0;
  for (int k = p.ch0; k < p.ch1; ++k, buf ^= 1) {
    fetch(k + 1);
    const float* one = s_bc[buf];
    float d[REGS], dx[REGS], ds[REGS], Bv[2][Lay::kBlock], Cv[2][Lay::kBlock];
    load_block<LN, NS, 0>(Bv[0], one);
    if constexpr (SEGS) load_block<LN, NS, 0>(Cv[0], one + kRows * P);
#pragma unroll
    for (int q = 0; q < REGS; ++q) {
      const float2 v = s_d[buf][mine][q * LN + l];
      d[q] = v.x, dx[q] = v.y;
      if constexpr (SEGS) ds[q] = s_ds[buf][mine][q * LN + l];
    }
    each<Lay::kBlocks>([&](auto K) {
      constexpr int b = K, R = Lay::kBlockRows;
      if constexpr (b + 1 < Lay::kBlocks) {
        load_block<LN, NS, b + 1>(Bv[(b + 1) % 2], one);
        if constexpr (SEGS) load_block<LN, NS, b + 1>(Cv[(b + 1) % 2], one + kRows * P);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (b % (Lay::kBlocks / MARKS) == 0) {
        constexpr int m = b / (Lay::kBlocks / MARKS), q0 = m * REGS / MARKS;
        store_states<NS>(marks.tile(k * MARKS + m, 1), moff, h);
        if constexpr (SEGS) {
          store_elem<float>(mark_sums.tile(k * MARKS + m, 1), on && l == 0 ? cm * 4 : kNowhere, steps);
          float sum = d[q0];
#pragma unroll
          for (int q = 1; q < REGS / MARKS; ++q) sum += d[q0 + q];
          steps += group_sum<LN>(sum);
        }
      }
      each<R>([&](auto J) {
        constexpr int j = b * R + J;
        const float dj = row_value<LN, NS, j>(d), dxj = row_value<LN, NS, j>(dx);
        float dsj = 0.f;
        if constexpr (SEGS) dsj = row_value<LN, NS, j>(ds);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const Decay<EXACT> e(dj * A2[s]);
          h[s] = e.of(h[s], dxj * Bv[b % 2][J * NS + s]);
          if constexpr (SEGS) {
            product[s] = e.of(product[s]);
            Q[s] = __builtin_fmaf(product[s], dsj * Cv[b % 2][J * NS + s], Q[s]);
          }
        }
      });
      pin_floats(h);
      if constexpr (SEGS) pin_floats(product), pin_floats(Q);
    });
    stage(buf ^ 1, k + 1);
    lds_barrier();
  }
  if (SEGS && on) {
    const size_t at = (((size_t)p.b * G.nseg + p.seg) * G.C + cm) * P + l * NS;
#pragma unroll
    for (int s = 0; s < NS; ++s) L.w.ends[at + s] = h[s], L.w.back[at + s] = Q[s];
    if (l == 0) L.w.steps[((size_t)p.b * G.nseg + p.seg) * G.C + cm] = steps;
  }
}

// two elements that a thread keeps, of bf16 in one register
template <typename T> struct Kept;
template <> struct Kept<bf16_t> {
  uint32_t w;
  __device__ __forceinline__ Kept() {}
  __device__ __forceinline__ Kept(uint32_t a, uint32_t b) : w(a | b << 16) {}
  __device__ __forceinline__ float first() const { return bf16_lo_half(w); }
  __device__ __forceinline__ float second() const { return bf16_hi_half(w); }
};
template <> struct Kept<float> {
  uint32_t a, b;
  __device__ __forceinline__ Kept() {}
  __device__ __forceinline__ Kept(uint32_t a, uint32_t b) : a(a), b(b) {}
  __device__ __forceinline__ float first() const { return __uint_as_float(a); }
  __device__ __forceinline__ float second() const { return __uint_as_float(b); }
};

// The gradients, chunk by chunk from the last one.
template <typename T, int LN, int NS, int THREADS, bool GATE>
__global__ __launch_bounds__(THREADS) CKDA_SCAN_BWD_WAVES(LN) void scan_bwd_kernel(const ScanLaunch L) {
  using Lay = Layout<LN, NS>;
  constexpr bool EXACT = sizeof(T) == 4;
  constexpr bool AHEAD = LN != 4;   // the next chunk's rows are loaded ahead (with 4 lanes other waves fill the wait)
  constexpr bool KEEP = NS <= 2;   // the decays of a chunk stay in registers; else they are formed twice
  constexpr int HALVES = Lay::kMarks, HR = kRows / HALVES;   // rows whose states are in registers at a time
  constexpr int CH = THREADS / LN, REGS = Lay::kRegs, P = Lay::kStates, WAVES = THREADS / 64;
  constexpr int PR = P / 16, kPart = kRows / 2 * PR * 64;   // a wave's dC and dB of a chunk: [row / 2][PR][lane]
  // (d, d x), then (d, u), of the same row and channel, which one wave reads and writes; ds, then s
  __shared__ float2 s_d[CH][kPad];
  __shared__ float s_ds[CH][kPad], s_v[CH][kPad];
  __shared__ __attribute__((aligned(16))) float s_bc[kRows * P * 2];
  __shared__ float s_part[WAVES][kPart];
  const SelScanArgs& a = L.a;
  const ScanGeom& G = L.G;
  ScanPlace p;
  if (!scan_place(L, p)) return;
  const int tid = threadIdx.x, l = tid % LN, mine = tid / LN;
  const int r = tid / CH, ch = tid % CH;
  const int c0 = p.cb * CH, first_c = p.g * G.Cg + c0;
  const bool on = c0 + mine < G.Cg, tile_on = c0 + ch < G.Cg;
  const int cm = first_c + mine, ct = first_c + ch;
  const size_t CN = (size_t)G.C * G.N;

  float A2[NS], Q[NS], start[NS], dA[NS];   // (A itself is A2 ln 2)
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int n = l * NS + s;
    const bool state = on && n < G.N;
    const size_t seg = (((size_t)p.b * G.nseg + p.seg) * G.C + cm) * P + n;
    A2[s] = state ? a.A[(size_t)cm * G.N + n] * kLog2e : 0.f;
    dA[s] = Q[s] = start[s] = 0.f;
    if (state) {
      if (G.nseg > 1) Q[s] = L.w.back[seg];
      else if (a.dhT) Q[s] = a.dhT[((size_t)p.b * G.C + cm) * G.N + n];
      if (p.seg > 0) start[s] = L.w.ends[seg];
    }
  }
  const float bias = tile_on && a.dt_bias ? a.dt_bias[ct] : 0.f;
  const float Dc = tile_on && a.D ? a.D[ct] : 0.f;
  float dD = 0.f, dbias = 0.f;

  const size_t first = (size_t)p.b * G.T;
  const Rows<T> xs(a.x, first, G.C), dts(a.dt, first, G.C), dys(a.dy, first, G.C), zs(a.z, first, G.ldz);
  const Rows<T> Bs(a.Bm, first, G.ldbc), Cs(a.Cm, first, G.ldbc);
  const Rows<T> dxs(a.dx, first, G.C), ddts(a.ddt, first, G.C), dzs(a.dz, first, G.C);
  const size_t first_mark = (size_t)p.b * G.chunks * HALVES;
  const Rows<float> marks(L.w.marks, first_mark, G.C * P), mark_sums(L.w.mark_steps, first_mark, G.C);
  int off[REGS], zoff[REGS];
#pragma unroll
  for (int i = 0; i < REGS; ++i) {
    off[i] = tile_on ? ((i * LN + r) * G.C + ct) * (int)sizeof(T) : kNowhere;
    zoff[i] = tile_on ? ((i * LN + r) * G.ldz + ct) * (int)sizeof(T) : kNowhere;
  }
  uint32_t xr[REGS], dr[REGS], zr[REGS] = {}, gr[REGS], mark[HALVES][NS], mark_steps[HALVES];
  BcTile<T, LN, NS, 1, THREADS, 3> bc;
  bc.place(L, p);
  auto fetch = [&](int chunk) {   // (before the segment's first chunk: nothing; no branch around the loads)
    const int row = chunk * kRows, rows = chunk >= p.ch0 ? min(p.len - row, kRows) : 0;
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      xr[i] = load_raw<T>(xs.tile(row, rows), off[i]);
      dr[i] = load_raw<T>(dts.tile(row, rows), off[i]);
      gr[i] = load_raw<T>(dys.tile(row, rows), off[i]);
      if (GATE) zr[i] = load_raw<T>(zs.tile(row, rows), zoff[i]);
    }
    bc.fetch(Bs, Cs, row, rows);
#pragma unroll
    for (int m = 0; m < HALVES; ++m) {
      load_states<NS>(mark[m], marks.tile(chunk * HALVES + m, rows > 0), on ? (cm * P + l * NS) * 4 : kNowhere);
      mark_steps[m] = load_raw<float>(mark_sums.tile(chunk * HALVES + m, p.seg > 0 && rows > 0), on ? cm * 4 : kNowhere);
    }
  };
  if (AHEAD && p.ch0 < p.ch1) fetch(p.ch1 - 1);
  for (int k = p.ch1 - 1; k >= p.ch0; --k) {
    const int row0 = k * kRows, rows = min(p.len - row0, kRows);
    if (!AHEAD) fetch(k);
    // the tile, and what its thread keeps of its rows for their outputs
    Kept<T> xd[REGS], zg[REGS];
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      xd[i] = Kept<T>(xr[i], dr[i]), zg[i] = Kept<T>(zr[i], gr[i]);
      float d = value_of<T>(dr[i]) + bias;
      if (G.softplus) d = softplus<EXACT>(d);
      d = tile_on && i * LN + r < rows ? d : 0.f;   // (dy, and so ds, is zero behind the rows)
      const float z = value_of<T>(zr[i]);
      s_d[ch][i * LN + r] = float2{d, d * value_of<T>(xr[i])};
      s_ds[ch][i * LN + r] = value_of<T>(gr[i]) * (GATE ? z * row_sigmoid<T>(z) : 1.f);
    }
    bc.stage(s_bc);
    float hc[HALVES][NS];   // the states before the chunk and its halves
#pragma unroll
    for (int m = 0; m < HALVES; ++m)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        hc[m][s] = value_of<float>(mark[m][s]);
        if (p.seg > 0) hc[m][s] += Decay<EXACT>(value_of<float>(mark_steps[m]) * A2[s]).of(start[s]);
      }
    lds_barrier();
    if (AHEAD) fetch(k - 1);
    float d[REGS], dx[REGS], ds[REGS];
#pragma unroll
    for (int q = 0; q < REGS; ++q) {
      const float2 v = s_d[mine][q * LN + l];
      d[q] = v.x, dx[q] = v.y;
      ds[q] = s_ds[mine][q * LN + l];
    }
    const float *Bl = s_bc, *Cl = s_bc + kRows * P;
    constexpr int BLK = Lay::kBlocks, R = Lay::kBlockRows;
    float Bv[2][Lay::kBlock], Cv[2][Lay::kBlock];   // of a block of rows, and of the next
    float* part = s_part[tid >> 6] + (tid & 63);
    each<HALVES>([&](auto Half) {
      constexpr int half = HALVES - 1 - Half, j0 = half * HR, b0 = half * BLK / HALVES, b1 = b0 + BLK / HALVES;
      Decay<EXACT> e[KEEP ? HR : 1][NS];
      float h[HR][NS], sums[LN], u[LN], v[LN], odd[PR];
      auto before = [&](int j, int s) { return j > j0 ? h[j - 1 - j0][s] : hc[half][s]; };
      load_block<LN, NS, b0>(Bv[b0 % 2], Bl);
      if constexpr (GATE) load_block<LN, NS, b0>(Cv[b0 % 2], Cl);
      each<BLK / HALVES>([&](auto K) {
        constexpr int b = b0 + K;
        if constexpr (b + 1 < b1) {
          load_block<LN, NS, b + 1>(Bv[(b + 1) % 2], Bl);
          if constexpr (GATE) load_block<LN, NS, b + 1>(Cv[(b + 1) % 2], Cl);
        }
        __builtin_amdgcn_sched_barrier(0);
        each<R>([&](auto J) {
          constexpr int j = b * R + J;
          const float dj = row_value<LN, NS, j>(d), dxj = row_value<LN, NS, j>(dx);
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const Decay<EXACT> now(dj * A2[s]);
            h[j - j0][s] = now.of(before(j, s), dxj * Bv[b % 2][J * NS + s]);
            if constexpr (KEEP) e[j - j0][s] = now;
            if constexpr (GATE) sums[j % LN] = s ? __builtin_fmaf(Cv[b % 2][J * NS + s], h[j - j0][s], sums[j % LN]) : Cv[b % 2][J * NS] * h[j - j0][s];
          }
        });
        if constexpr (GATE && (b + 1) * R % LN == 0) s_ds[mine][(b + 1) * R - LN + l] = turn_lanes<LN>(sums, l);
      });
      pin_floats(d), pin_floats(dx);   // (the broadcasts below are made again where they are used, not kept from above)
      load_block<LN, NS, b1 - 1>(Bv[(b1 - 1) % 2], Bl);
      load_block<LN, NS, b1 - 1>(Cv[(b1 - 1) % 2], Cl);
      each<BLK / HALVES>([&](auto K) {
        constexpr int b = b1 - 1 - K;
        if constexpr (b > b0) {
          load_block<LN, NS, b - 1>(Bv[(b + 1) % 2], Bl);
          load_block<LN, NS, b - 1>(Cv[(b + 1) % 2], Cl);
        }
        __builtin_amdgcn_sched_barrier(0);
        each<R>([&](auto J) {
          constexpr int i = R - 1 - J, j = b * R + i;
          const float dj = row_value<LN, NS, j>(d), dxj = row_value<LN, NS, j>(dx), dsj = row_value<LN, NS, j>(ds);
          float dC[NS], dB[NS];
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const float R_ = __builtin_fmaf(dsj, Cv[b % 2][i * NS + s], Q[s]);
            dC[s] = dsj * h[j - j0][s], dB[s] = dxj * R_;
            u[j % LN] = s ? __builtin_fmaf(R_, Bv[b % 2][i * NS + s], u[j % LN]) : R_ * Bv[b % 2][i * NS];
            Q[s] = KEEP ? e[KEEP ? j - j0 : 0][s].of(R_) : Decay<EXACT>(dj * A2[s]).of(R_);
            const float q = Q[s] * before(j, s);
            v[j % LN] = s ? __builtin_fmaf(q, A2[s], v[j % LN]) : q * A2[0];
            dA[s] = __builtin_fmaf(q, dj, dA[s]);
          }
          // dC and dB of the wave's channels: in the halves of the wave, two rows in their halves, states in the quads
          float both[PR];
          if constexpr (LN == 4) {
            float sc, sb;
            sum_quads(dC, dB, sc, sb);
            both[0] = sum_halves(sc, sb);
          } else {
#pragma unroll
            for (int s = 0; s < NS; ++s) both[s] = sum_halves(dC[s], dB[s]);
          }
#pragma unroll
          for (int s = 0; s < PR; ++s) {
            if constexpr (j % 2) odd[s] = both[s];
            else part[(j / 2 * PR + s) * 64] = sum_quarters(both[s], odd[s]);
          }
        });
        pin_floats(Q), pin_floats(dA);
        if constexpr (b * R % LN == 0) {   // LN rows done: lane l has those of row b R + l
          s_d[mine][b * R + l].y = turn_lanes<LN>(u, l);
          s_v[mine][b * R + l] = turn_lanes<LN>(v, l) * kLn2;
        }
      });
    });
    lds_barrier();
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      const float2 du = s_d[ch][i * LN + r];
      const float x = xd[i].first(), dy = zg[i].second(), z = zg[i].first();
      const float sg = GATE ? row_sigmoid<T>(z) : 0.f, dsr = GATE ? dy * z * sg : dy;
      const float dd = __builtin_fmaf(x, du.y, s_v[ch][i * LN + r]);
      const float ddt = G.softplus ? dd * softplus_slope<EXACT>(xd[i].second() + bias) : dd;
      store_elem<T>(dxs.tile(row0, rows), off[i], __builtin_fmaf(Dc, dsr, du.x * du.y));
      store_elem<T>(ddts.tile(row0, rows), off[i], ddt);
      if constexpr (GATE)
        store_elem<T>(dzs.tile(row0, rows), off[i], dy * __builtin_fmaf(Dc, x, s_ds[ch][i * LN + r]) * silu_slope(z, sg));
      dD = __builtin_fmaf(dsr, x, dD);
      dbias += i * LN + r < rows ? ddt : 0.f;
    }
    // dC (lower half of a wave's lanes) and dB of the workgroup's channels; odd DPP rows hold the second of two rows
#pragma unroll
    for (int i = 0; i < kPart / THREADS; ++i) {
      const int at = tid + i * THREADS, lane = at % 64, which = lane / 32, t = at / (64 * PR) * 2 + (lane / 16 & 1);
      const int bank = lane / 4 % 4;
      const int n = LN == 4 ? lane % 4 * 4 + (bank & 1) * 2 + bank / 2 : lane % 16 * NS + at / 64 % PR;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) sum += s_part[w][at];
      if (t < rows && n < G.N)
        L.w.bc[((((size_t)p.g * G.cblocks + p.cb) * G.B + p.b) * G.T + row0 + t) * 2 * G.N + which * G.N + n] = sum;
    }
    lds_barrier();   // the next chunk's tile goes to the same place
  }
  float* part = L.w.weights + ((size_t)p.b * G.nseg + p.seg) * (CN + 2 * (size_t)G.C);
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int n = l * NS + s;
    if (!on || n >= G.N) continue;
    part[(size_t)cm * G.N + n] = dA[s];
    if (p.seg == 0 && a.dh0) a.dh0[((size_t)p.b * G.C + cm) * G.N + n] = Q[s];
  }
  // over the tile's rows: thread (r, ch) holds the sums of rows r, r + LN, ...
  s_ds[ch][r] = dD;
  s_v[ch][r] = dbias;
  __syncthreads();
  if (tid < 2 * CH && c0 + tid % CH < G.Cg) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < LN; ++i) sum += tid < CH ? s_ds[tid % CH][i] : s_v[tid % CH][i];
    part[CN + (size_t)(tid / CH) * G.C + first_c + tid % CH] = sum;
  }
  if (G.pad_zero && tile_on) {
    const T zero = from_f32<T>(0.f);
    const int to = (int)min(((long long)p.ch0 + G.seg_chunks) * kRows, (long long)G.T);
    for (int t = max(p.len, p.ch0 * kRows) + r; t < to; t += LN) {
      const size_t at = ((size_t)p.b * G.T + t) * G.C + ct;
      ((T*)a.dx)[at] = ((T*)a.ddt)[at] = zero;
      if (GATE) ((T*)a.dz)[at] = zero;
    }
  }
}

// dBm and dCm, the sums of the channel blocks' parts, by the first workgroups, and the
// weights' gradients by the others (one launch: 4 us less than two)
template <typename T>
__global__ __launch_bounds__(256) void scan_sums_kernel(const ScanLaunch L, const SumOuts weights, unsigned first) {
  if (blockIdx.x >= first) {
    sum_parts<256 / kSumCols>(weights, blockIdx.x - first);
    return;
  }
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
    if (G.softplus) d = softplus<EXACT>(d);
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

// (the forward with 16 lanes: 16 channels a workgroup; MI355X, us, with 8, 16 and 32: B4 T4096 C2048 237, 233 and
// 243, of 64 states 261, 221 and 270)
constexpr int kFwdThreads = 256;                       // of every layout
constexpr int kQuadThreads = 256, kWideThreads = 512;   // of the backward's passes

// How a call runs: lanes and states a channel, channels of a workgroup, segments.
struct ScanPlan {
  ScanGeom G;
  int ln, ns;
};
ScanPlan scan_plan(int B, int T, int C, int G, int N, bool bwd) {
  ScanPlan plan = {};
  ScanGeom& g = plan.G;
  g.B = B, g.T = T, g.C = C, g.G = G, g.N = N;
  g.Cg = C / G;
  g.chunks = (int)(((long long)T + kRows - 1) / kRows);
  // 4 lanes a channel where that can fill three waves of every SIMD, by segments of 128 rows or more; but in the
  // forward not where 16 lanes fill two without segments and 4 lanes would need them, which cost a pass of their own
  // (MI355X, us, 4 and 16 lanes: forward B4 T4096 C2048 257 and 213, B16 T1024 C4096 279 and 315, B1 T32768 C1024 257
  // and 299, B1 T1024 C1024 36 and 22; backward B4 T4096 C2048 632 and 855, fp32 B3 T777 C500 149 and 90).  The two
  // meet at some 6000 channels, below the 8192 that fill two waves (forward B4 T4096, 4 and 16 lanes: C1920 258 and
  // 213, C1536 216 and 212, C1024 134 and 143, C512 76 and 82; fp32 C2048 443 and 367, C1920 458 and 365, C1024 231
  // and 243): between, the rule takes the slower one.
  const long long channels = (long long)B * C, blocks4 = (long long)B * G * ((g.Cg + 63) / 64);
  const bool fills = blocks4 * std::max(1, g.chunks / 8) >= 768, alone = !bwd && channels >= 8192 && channels < 49152;
  const bool quad = N <= 16 && fills && !alone;
  plan.ln = quad ? 4 : 16;
  plan.ns = quad ? 4 : N <= 16 ? 1 : N <= 32 ? 2 : 4;
  const int ch = (quad ? kQuadThreads : bwd ? kWideThreads : kFwdThreads) / plan.ln;
  g.cblocks = (g.Cg + ch - 1) / ch;
  // Segments where the channels leave SIMDs without waves (fewer than three with 4 lanes, two with 16): four then.
  // The backward's main pass with 4 lanes keeps three: two rounds of those (B4 T4096 C2048: 632, and with 1024
  // workgroups, a round and a third, 644).
  const long long blocks = (long long)B * G * g.cblocks, full = !quad ? 16384 / ch : bwd ? 1536 : 1024;
  g.nseg = 1;
  if (blocks > 0 && blocks < (quad ? 768 : full * 3 / 8))
    g.nseg = (int)std::max(1LL, std::min((full + blocks - 1) / blocks, (long long)g.chunks / 8));
  g.seg_chunks = std::max(1, (g.chunks + g.nseg - 1) / g.nseg);
  g.nseg = std::max(1, (g.chunks + g.seg_chunks - 1) / g.seg_chunks);
  return plan;
}

struct ScanSizes {
  size_t ends, steps, back, marks, mark_steps, bc, weights;   // floats
};
ScanSizes scan_sizes(const ScanPlan& plan, bool bwd) {
  auto up = [](size_t n) { return (n + 63) / 64 * 64; };
  const ScanGeom& g = plan.G;
  const size_t CP = (size_t)g.C * plan.ln * plan.ns, segs = (size_t)g.B * g.nseg;
  ScanSizes s = {};
  if (g.nseg > 1) s.ends = up(segs * CP), s.steps = up(segs * g.C);
  if (!bwd) return s;
  const size_t marks = (size_t)g.chunks * (plan.ln == 4 ? Layout<4, 4>::kMarks : 1);
  if (g.nseg > 1) s.back = up(segs * CP), s.mark_steps = up((size_t)g.B * marks * g.C);
  s.marks = up((size_t)g.B * marks * CP);
  s.bc = up((size_t)g.G * g.cblocks * g.B * g.T * 2 * g.N);
  s.weights = up(segs * ((size_t)g.C * g.N + 2 * (size_t)g.C));
  return s;
}
size_t scan_bytes(const ScanSizes& s) {
  return 4 * (s.ends + s.steps + s.back + s.marks + s.mark_steps + s.bc + s.weights);
}

ScanLaunch scan_launch(const SelScanArgs& a, const ScanPlan& plan, bool bwd) {
  ScanLaunch L;
  L.a = a;
  L.G = plan.G;
  L.G.ldbc = a.ldbc, L.G.ldz = a.ldz, L.G.softplus = a.softplus, L.G.pad_zero = a.pad_zero;
  L.segs = L.G.nseg;
  const ScanSizes s = scan_sizes(plan, bwd);
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

hipError_t launch_join(const ScanLaunch& L, int P, bool bwd) {
  const unsigned half = (unsigned)(((long long)L.G.B * L.G.C * P + 255) / 256), blocks = bwd ? 2 * half : half;
  if (L.a.dtype == CKDA_DTYPE_F32) hipLaunchKernelGGL(scan_join_kernel<true>, dim3(blocks), dim3(256), 0, L.a.stream, L, P, half);
  else hipLaunchKernelGGL(scan_join_kernel<false>, dim3(blocks), dim3(256), 0, L.a.stream, L, P, half);
  return hipGetLastError();
}

template <typename T, int LN, int NS> hipError_t launch_fwd_t(const SelScanArgs& a, const ScanPlan& plan) {
  constexpr int SUBS = LN == 4 ? 1 : 2;   // a tile of 64 channels and 16 rows, or 16 and 32
  ScanLaunch L = scan_launch(a, plan, false);
  if (L.G.nseg > 1) {
    L.segs = L.G.nseg - 1;
    hipLaunchKernelGGL((scan_fwd_kernel<T, LN, NS, kFwdThreads, SUBS, false>), dim3(scan_blocks(L)), dim3(kFwdThreads), 0, a.stream, L);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = launch_join(L, LN * NS, false);
    if (e != hipSuccess) return e;
    L.segs = L.G.nseg;
  }
  hipLaunchKernelGGL((scan_fwd_kernel<T, LN, NS, kFwdThreads, SUBS, true>), dim3(scan_blocks(L)), dim3(kFwdThreads), 0, a.stream, L);
  return hipGetLastError();
}

template <typename T, int LN, int NS> hipError_t launch_bwd_t(const SelScanArgs& a, const ScanPlan& plan) {
  constexpr int THREADS = LN == 4 ? kQuadThreads : kWideThreads;
  const ScanLaunch L = scan_launch(a, plan, true);
  const dim3 grid(scan_blocks(L)), block(THREADS);
  hipError_t e = hipSuccess;
  if (L.G.B > 0 && L.G.C > 0) {
    if (L.G.nseg > 1) {
      hipLaunchKernelGGL((scan_prep_kernel<T, LN, NS, THREADS, true>), grid, block, 0, a.stream, L);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      if ((e = launch_join(L, LN * NS, true)) != hipSuccess) return e;
    } else {
      hipLaunchKernelGGL((scan_prep_kernel<T, LN, NS, THREADS, false>), grid, block, 0, a.stream, L);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.z) hipLaunchKernelGGL((scan_bwd_kernel<T, LN, NS, THREADS, true>), grid, block, 0, a.stream, L);
    else hipLaunchKernelGGL((scan_bwd_kernel<T, LN, NS, THREADS, false>), grid, block, 0, a.stream, L);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const long long each = (long long)a.B * a.T * 2 * a.G * a.N;
  const unsigned first = (unsigned)((each + 255) / 256);
  const size_t CN = (size_t)a.C * a.N, C = (size_t)a.C;
  const SumOuts weights = sum_outs(PartSums{L.w.weights, L.G.B * L.G.nseg, CN + 2 * C, {a.dA, a.dD, a.dbias}, {CN, C, C}});
  const unsigned blocks = first + (wanted(weights) ? sum_blocks(weights) : 0);   // (without channels dB and dC are zeros)
  if (blocks == 0) return e;
  hipLaunchKernelGGL((scan_sums_kernel<T>), dim3(blocks), dim3(256), 0, a.stream, L, weights, first);
  return hipGetLastError();
}

// Two sequences a thread where that leaves threads enough (MI355X, us, one and two: 256 sequences of 4096 channels
// with 16 states 32.5 and 28, 64 of 2048 with 64 states 18.6 and 16).
template <typename T, int LPC, bool WHOLE> hipError_t launch_decode_t(const SelScanArgs& a) {
  const ScanLaunch L = scan_launch(a, scan_plan(a.B, a.T, a.C, a.G, a.N, false), false);
  const bool many = (long long)a.B * a.C * LPC >= 1 << 20;
  const long long groups = many ? ((long long)a.B + 1) / 2 : a.B;
  const unsigned blocks = (unsigned)((groups * a.C * LPC + 255) / 256);
  if (many) hipLaunchKernelGGL((scan_decode_kernel<T, LPC, WHOLE, 2>), dim3(blocks), dim3(256), 0, a.stream, L);
  else hipLaunchKernelGGL((scan_decode_kernel<T, LPC, WHOLE, 1>), dim3(blocks), dim3(256), 0, a.stream, L);
  return hipGetLastError();
}

template <typename T> hipError_t launch_scan_fwd_t(const SelScanArgs& a) {
  const ScanPlan plan = scan_plan(a.B, a.T, a.C, a.G, a.N, false);
  if (plan.ln == 4) return launch_fwd_t<T, 4, 4>(a, plan);
  if (plan.ns == 1) return launch_fwd_t<T, 16, 1>(a, plan);
  return plan.ns == 2 ? launch_fwd_t<T, 16, 2>(a, plan) : launch_fwd_t<T, 16, 4>(a, plan);
}
template <typename T> hipError_t launch_scan_bwd_t(const SelScanArgs& a) {
  const ScanPlan plan = scan_plan(a.B, a.T, a.C, a.G, a.N, true);
  if (plan.ln == 4) return launch_bwd_t<T, 4, 4>(a, plan);
  if (plan.ns == 1) return launch_bwd_t<T, 16, 1>(a, plan);
  return plan.ns == 2 ? launch_bwd_t<T, 16, 2>(a, plan) : launch_bwd_t<T, 16, 4>(a, plan);
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
  return scan_bytes(scan_sizes(scan_plan(B, T, C, G, N, false), false));
}
size_t scan_bwd_workspace_bytes(int B, int T, int C, int G, int N) {
  return scan_bytes(scan_sizes(scan_plan(B, T, C, G, N, true), true));
}

// fewer than 2^32 threads in every launch, and counts of workgroups in an int
bool scan_fits_grid(int B, int T, int C, int G, int N) {
  const ScanGeom g = scan_plan(B, T, C, G, N, true).G, f = scan_plan(B, T, C, G, N, false).G;
  const long long groups = (long long)B * G;
  return groups * g.nseg * g.cblocks < (1LL << 22) && groups * f.nseg * f.cblocks < (1LL << 22) &&
         (long long)B * C * 64 < (1LL << 31) && (double)B * T * 2 * G * N + 256.0 / kSumCols * (N + 2.0) * C < 4e9;
}

hipError_t launch_scan_fwd(const SelScanArgs& a) {
  return a.dtype == CKDA_DTYPE_BF16 ? launch_scan_fwd_t<bf16_t>(a) : launch_scan_fwd_t<float>(a);
}
hipError_t launch_scan_bwd(const SelScanArgs& a) {
  return a.dtype == CKDA_DTYPE_BF16 ? launch_scan_bwd_t<bf16_t>(a) : launch_scan_bwd_t<float>(a);
}
hipError_t launch_scan_decode(const SelScanArgs& a) {
  return a.dtype == CKDA_DTYPE_BF16 ? launch_decode<bf16_t>(a) : launch_decode<float>(a);
}

}  // namespace ckda
