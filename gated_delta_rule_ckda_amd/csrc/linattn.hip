// linattn.hip -- linear attention with a decay for each head: the chunked
// sweep behind the forward and the three gradient sweeps of the backward.
//
// One independent state per (batch, head), a_t = exp(g_t):
//   H_t = a_t H_{t-1} + k_t v_t^T,   o_t = H_t^T q_t.
// Over a chunk of C = 64 rows with c_t = g_1 + ... + g_t (inside the chunk)
// and G(t, s) = exp(c_t - c_s), H the state before the chunk:
//   o_t = exp(c_t) H^T q_t + sum_{s <= t} G(t, s) (q_t . k_s) v_s
//   H  <- exp(c_C) H + sum_s G(C, s) k_s v_s^T.
// The gradients are the same recurrence with the roles of the vectors turned
// (R_t = dL/dH_t, R_t = a_{t+1} R_{t+1} + q_t do_t^T, R_T = dhT + q_T do_T^T):
//   dq_t = H_t do_t     reads H^T  = sum v k^T   forward in time,
//   dk_t = R_t v_t      reads R^T  = sum do q^T  backward in time,
//   dv_t = R_t^T k_t    reads R    = sum q do^T  backward in time,
// and dh0 = a_1 R_1.  A sweep backward in time is a sweep over the reversed
// rows whose row j has the decay of row j - 1 (the first has none).  So one
// kernel serves all four: a "sweep" has an x operand (its queries), a y
// operand (its keys), a z operand (its values) and a state [D1, D2].
//
// One workgroup runs one slice of DS value columns of one (batch, head) over
// one segment of rows; the columns of the state evolve independently, and the
// state slice never leaves the workgroup.  Eight waves: four "output waves",
// each with 16 of the chunk's 64 rows, and four "state waves" that carry the
// state slice in their accumulators and bring the next chunk's operands into
// LDS.  A chunk has two phases with a barrier after each:
//   1  output waves read H, Y and Z from LDS and multiply: S^T = Y X^T tile by
//      tile (rows s, columns t) and H^T X^T; state waves read the columns of Y
//      and of G(C, .) Z and form the next chunk's decay factors;
//   2  output waves: P^T = G . S^T in fp32 on the accumulators, which are then,
//      in the K order of ckda_device.hpp, the B operand of Z^T P^T; exp(c_t)
//      scales the accumulators of H^T X^T (a factor of the column); outputs.
//      State waves: H <- exp(c_C) H + Y^T (G(C, .) Z); the new H^T, and Y, Z
//      and the terms of G(C, .) Z of the next chunk into the same LDS buffers.
// Precision: the inputs are exact in bf16; every factor that is not (P, H and
// the scaled Z) is carried as a sum of bf16 terms: two (16 bits) where the
// product ends in a rounded output, three (24 bits) for the state itself,
// which is returned in fp32 (two where none is).  All sums are fp32.  fp32
// inputs take the fp32 matrix cores throughout.
// What bounds it (MI355X, bf16, d128): with slices of 32 columns each CU's
// vector-memory return path, 84% busy (TD_TD_BUSY) at some 11 bytes a cycle, as
// every slice reads the chunk's x and y again (B4 H16 T4096, 256 workgroups: 104
// us, 260 MB of HBM traffic); with whole states of 128 columns no unit by itself
// (the backward's three sweeps of that size, 192 workgroups: 245 us, 810 MB;
// return path 57%, matrix cores 21%, LDS 27% busy): one workgroup to a CU waits at
// two barriers a chunk; in short calls the latency of the first loads and of a
// chunk's two phases (77 rows: 6.8 us).  fp32: that latency too (B3 H8 T1000 dk64
// dv128: 38 us, matrix cores 18%, return path 24% busy).
// Log decays are summed as two parts, whole multiples of 1/64 (whose sums are
// exact) and the rest, so that differences of large sums keep fp32 accuracy.
// (g log2 e itself is rounded once for each row, by 2^-24 of it: at most 4e-8 of
// the norm of o over 1000 rows of constant decays, the products' own roundings
// being 2e-7.)
#include <algorithm>
#include <type_traits>

#include "ckda_device.hpp"
#include "ckda_internal.hpp"

namespace ckda {

namespace {

constexpr int C = kLaChunk;    // rows of a chunk
constexpr int RT = C / 16;     // row tiles
// decay factors of a chunk's rows: c (whole part), c (rest), exp(c_t), G(C, t),
// G(e, t) with e the last row of t's tile
constexpr int kDecSets = 5;
constexpr int kDecFloats = kDecSets * C + 4;   // and, behind them, the chunk's decay less 1 (or 0: decay_step)

template <typename T, int D1, int DS, bool EXACT>
struct SweepCfg {
  static constexpr int E = (int)sizeof(T);
  static constexpr bool BF = E == 2;
  static constexpr int KB = FragTraits<T>::KB;
  static constexpr int D1P = D1 < KB ? KB : D1;      // contraction width, whole K blocks
  static constexpr int KBN = D1P / KB;               // K blocks over D1
  static constexpr int KBC = C / KB;                 // K blocks over the chunk's rows
  static constexpr int RH = D1 / 16;                 // state row tiles
  static constexpr int NDV = DS / 16;                // state column tiles of the slice
  static constexpr int YROW = D1P * E, ZROW = DS * E;   // bytes of a row in LDS
  // four state waves on WR x WC blocks of TR x TC state tiles
  static constexpr int WC = RH == 1 ? (NDV < 4 ? NDV : 4) : (NDV == 1 ? 1 : 2), WR = 4 / WC;
  static constexpr int TR = (RH + WR - 1) / WR, TC = NDV / WC;
  static constexpr int Y_BYTES = C * YROW, Z_BYTES = C * ZROW, H_BYTES = DS * YROW;
  static constexpr int HSETS = BF ? 2 : 1;           // terms of H: hi and lo
  static constexpr int ZSETS = BF ? (EXACT ? 3 : 2) : 1;   // terms of the scaled Z
  // LDS: Y, Z, the terms of G(C, .) Z, the terms of H^T, two sets of decay factors
  static constexpr int Z_OFF = Y_BYTES, ZS_OFF = Z_OFF + Z_BYTES, H_OFF = ZS_OFF + ZSETS * Z_BYTES;
  static constexpr int DEC_OFF = H_OFF + HSETS * H_BYTES, DEC_BYTES = kDecFloats * 4;
  static constexpr int LDS_BYTES = DEC_OFF + 2 * DEC_BYTES;
  // Pieces of 16 bytes to copy, in units of one piece for each of 256 threads:
  // by the state waves, but for the first YO units of Y and ZO of Z of the
  // widest slices, which the output waves copy (a unit of Z costs some ten
  // times one of Y, for its scaled terms).  Units are loaded NR chunks before
  // they are copied; a chunk of a narrow slice takes less time than a load, and
  // the widest have no registers for two (fp32 128 x 64, B8 H32 T512: forward 143
  // us, 194 with two and 85 registers spilled; backward 432 and 567).
  static constexpr int YPR = D1 * E / 16, ZPR = ZROW / 16;
  static constexpr int NY = (C * YPR + 255) / 256, NZ = (C * ZPR + 255) / 256;
  static constexpr int YO = DS == 128 ? NY / 2 : 0, ZO = DS == 128 ? NZ / 4 : 0;
  static constexpr int NR = DS == 128 || D1 * DS * E >= 32768 ? 1 : 2;
};

// Byte offset of the 16-byte piece `piece` of row `row` in an LDS array of
// ROWB-byte rows.  The piece index is xor-ed with twice the number of the
// row's 256-byte line, so that neither kind of operand read has bank conflicts
// (SQ_LDS_BANK_CONFLICT 0 in own_state_kernel; the sweeps' conflicts, 10 to 15% of
// their LDS cycles at d128, are those of other accesses): a transposing 8-byte read takes 32 bytes of 8 rows
// at a time, a 16-byte read of 16 rows takes rows 0-3 and 12-15 of one piece
// with rows 4-11 of the next.  (Telling rows r and r + 8 apart as well costs
// the 16-byte reads a two-way conflict.)
template <int ROWB>
__device__ __forceinline__ int lds_piece(int row, int piece) {
  constexpr int NCH = ROWB / 16 < 16 ? ROWB / 16 : 16;
  const int i = row / (16 / NCH);
  const int s = (i & (NCH / 2 - 1)) << 1;
  return row * ROWB + ((piece ^ s) << 4);
}

// The same for the H^T arrays, which are read as rows like Y but written in
// 8-byte halves of one piece of 16 rows: with 256-byte rows these then fall on
// different banks too.
template <int ROWB>
__device__ __forceinline__ int state_piece(int row, int piece) {
  if constexpr (ROWB == 256) return row * ROWB + ((piece ^ ((row & 15) ^ (((row >> 2) ^ (row >> 3)) & 1))) << 4);
  else return lds_piece<ROWB>(row, piece);
}

// Operand reads.  A lane's address is kept as one offset for each piece or
// column tile, opaque to the compiler (it would otherwise keep one for every
// read, as the constants beside it pass the 16-bit offsets of LDS
// instructions); row tiles, K blocks and terms are constant distances from it.
// 16-byte pieces of row r of a row tile, K block kb along the row; base: the array's offset
template <int ROWB, int KBN, bool STATE>
struct RowFrags {
  int off[KBN];
  __device__ __forceinline__ RowFrags(int base, int g, int r) {
#pragma unroll
    for (int kb = 0; kb < KBN; ++kb) {
      off[kb] = base + (STATE ? state_piece<ROWB>(r, kb * 4 + g) : lds_piece<ROWB>(r, kb * 4 + g));
      asm("" : "+v"(off[kb]));
    }
  }
  __device__ __forceinline__ Frag read(const unsigned char* lds, int tile, int kb, int beyond = 0) const {
    return load_frag(lds + off[kb] + tile * 16 * ROWB + beyond);
  }
};

// column col0 + r, rows of K block kb in the K order kappa
template <typename T, int ROWB>
struct ColFrags {
  static constexpr bool BF = sizeof(T) == 2;
  int off[BF ? 1 : 4];
  __device__ __forceinline__ void set(int base, int col0, int g, int r) {
    if constexpr (BF) {
      // two transposing reads (ds_read_b64_tr_b16): within 16 lanes, lane i gets
      // as element j the element i % 4 of the 8 bytes lane 4 j + i / 4 addresses
      off[0] = base + lds_piece<ROWB>(4 * g + (r >> 2), col0 / 8 + ((r & 3) >> 1)) + (r & 1) * 8;
      asm("" : "+v"(off[0]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        off[e] = base + lds_piece<ROWB>(4 * g + e, (col0 + r) / 4) + ((col0 + r) % 4) * 4;
        asm("" : "+v"(off[e]));
      }
    }
  }
  __device__ __forceinline__ Frag read(const unsigned char* lds, int kb, int beyond = 0) const {
    Frag f;
    if constexpr (BF) {
      typedef short v4s __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4s lds_v4s;
      const unsigned char* p = lds + off[0] + kb * 32 * ROWB + beyond;   // (16 rows on: the same piece order)
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p));
      const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 16 * ROWB)));
      f.w = u32x4{a[0], a[1], b[0], b[1]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        f.w[e] = *reinterpret_cast<const uint32_t*>(lds + off[e] + kb * 16 * ROWB + beyond);
    }
    return f;
  }
};

// inclusive prefix sum over the wave's 64 lanes (DPP row shifts, then the
// last lane of each row into the rows after it)
__device__ __forceinline__ float wave_prefix(float x) {
#define CKDA_STEP(CTRL, ROWS) \
  x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, false))
  CKDA_STEP(0x111, 0xF);   // row_shr:1
  CKDA_STEP(0x112, 0xF);   // row_shr:2
  CKDA_STEP(0x114, 0xF);   // row_shr:4
  CKDA_STEP(0x118, 0xF);   // row_shr:8
  CKDA_STEP(0x142, 0xA);   // row_bcast:15 into rows 1 and 3
  CKDA_STEP(0x143, 0xC);   // row_bcast:31 into rows 2 and 3
#undef CKDA_STEP
  return x;
}

// sum over this lane and those after it (row_shl within rows, then the sums of the rows after)
__device__ __forceinline__ float wave_suffix(float x, int lane) {
#define CKDA_STEP(CTRL) \
  x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false))
  CKDA_STEP(0x101);
  CKDA_STEP(0x102);
  CKDA_STEP(0x104);
  CKDA_STEP(0x108);
#undef CKDA_STEP
  auto first = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l)); };
  const float s3 = first(48), s2 = first(32) + s3, s1 = first(16) + s2;
  return x + (lane < 16 ? s1 : lane < 32 ? s2 : lane < 48 ? s3 : 0.f);
}
// the value of the lane before this one (DPP wave_shr), 0 for the first
__device__ __forceinline__ float lane_before(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x138, 0xF, 0xF, false));
}

// the value of lane 15 of this lane's row of 16 (DPP row_newbcast)
__device__ __forceinline__ float row_last(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x15F, 0xF, 0xF, false));
}

// sum over the lanes r, r + 16, r + 32 and r + 48 (in pairs of rows, then of
// halves: both operands of a swap the same register)
__device__ __forceinline__ float row_groups_sum(float x) {
  const uint32_t a = __float_as_uint(x);
  const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t b = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kDecayFloor = -240.f;   // 2^-240 is 0 in fp32, and 64 such steps keep their sum's parts exact

// x less the low / high half of a packed bf16 pair, exact where x - half is a
// float (a residual always is): one dot product with (-1, 0) / (0, -1) instead
// of widening the half and subtracting it.  (The constant sits in a register:
// as a literal of the packed instruction it gave wrong sums.)
__device__ __forceinline__ float less_half(float x, uint32_t pair, uint32_t minus_one) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  asm("" : "+s"(minus_one));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, minus_one), x, false);
}
constexpr uint32_t kMinusLo = 0x0000BF80u, kMinusHi = 0xBF800000u;   // (-1, 0), (0, -1) in bf16

// the two terms of the pair (a, b), packed: hi + lo = x to 2^-16 of |x|
__device__ __forceinline__ void split2(float a, float b, uint32_t& h, uint32_t& l) {
  h = pack_bf16x2(a, b);
  asm("" : "+v"(h));
  l = pack_bf16x2(less_half(a, h, kMinusLo), less_half(b, h, kMinusHi));
}
// N = 2 or 3 terms of eight values: their sum is x to 2^-16 or 2^-25 of |x|
template <int N>
__device__ __forceinline__ void split_terms(const float* v, Frag* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t h = pack_bf16x2(a, b);
      asm("" : "+v"(h));
      f[n].w[i] = h;
      if (n + 1 < N) {
        a = less_half(a, h, kMinusLo);
        b = less_half(b, h, kMinusHi);
      }
    }
  }
}

// A slow decay of a chunk (or segment), applied again and again to a long memory,
// has to keep its distance from 1: as a float near 1 it is off by 2^-24 and more
// with every chunk, always to the same side where the decay is constant.  It is
// held as 2^x - 1, a polynomial (the series of e^y - 1 up to y^7, |y| < 0.35, off by
// 2e-8 of it), and applied by one multiply-add; 0 where 2^x itself will do.
// (Decays of exactly 1 are 0 too.)
__device__ __forceinline__ float decay_less_one(float x) {
  const float y = x * 0.6931471805599453f;
  float p = 1.f / 5040.f;
  p = __builtin_fmaf(p, y, 1.f / 720.f);
  p = __builtin_fmaf(p, y, 1.f / 120.f);
  p = __builtin_fmaf(p, y, 1.f / 24.f);
  p = __builtin_fmaf(p, y, 1.f / 6.f);
  p = __builtin_fmaf(p, y, 0.5f);
  p = __builtin_fmaf(p, y, 1.f);
  return fabsf(x) < 0.5f ? p * y : 0.f;
}
// the decayed state: `end` and `less` of a chunk, the same for all lanes
template <int TR, int TC>
__device__ __forceinline__ void decay_step(f32x4 (&h)[TR][TC], float end, float less) {
  if (__builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, less)) != 0) {
#pragma unroll
    for (int i = 0; i < TR; ++i)
#pragma unroll
      for (int j = 0; j < TC; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) h[i][j][e] = __builtin_fmaf(h[i][j][e], less, h[i][j][e]);
  } else {
#pragma unroll
    for (int i = 0; i < TR; ++i)
#pragma unroll
      for (int j = 0; j < TC; ++j) h[i][j] *= end;
  }
}

// Decay factors of a chunk from the log decays g (one row a lane) into dec;
// drop: the chunk's rows are to have no part in the state after it.
__device__ __forceinline__ void decay_factors(float g, float* dec, int lane, bool drop = false) {
  float x = g * kLog2E;
  x = x < kDecayFloor ? kDecayFloor : x;   // keeps NaN
  const float whole = rintf(x * 64.f) * (1.f / 64.f);
  const float ch = wave_prefix(whole), cl = wave_prefix(x - whole);
  const float th = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ch), 63));
  const float tl = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, cl), 63));
  dec[lane] = ch;
  dec[C + lane] = cl;
  dec[2 * C + lane] = __builtin_amdgcn_exp2f(ch + cl);
  dec[3 * C + lane] = drop ? 0.f : __builtin_amdgcn_exp2f((th - ch) + (tl - cl));
  dec[4 * C + lane] = __builtin_amdgcn_exp2f((row_last(ch) - ch) + (row_last(cl) - cl));
  if (lane == 0) dec[kDecSets * C] = decay_less_one(th + tl);
}

// The rows a workgroup works on: chunk row j of a segment is row row0 + j of
// the sweep, which is that row of the sequence, or the up - 1 - that one, up
// being len rounded up to whole chunks: the chunks of both directions are the
// same rows (decay_grad_kernel adds what their sweeps leave chunk by chunk).
// Rows outside [0, len) fall outside the buffers: they read as zero and are
// not stored.
struct Rows {
  int len, up, row0, nch, last, dir, first;
  __device__ __forceinline__ Rows(const SweepLaunch& L, int bh, int seg, int seg_rows, int reverse) {
    len = L.lens ? min(max(L.lens[bh / L.heads], 0), L.rows) : L.rows;
    up = (len + C - 1) / C * C;
    row0 = seg * seg_rows;
    nch = (min(max(len - row0, 0), seg_rows) + C - 1) / C;
    last = max(nch - 1, 0);
    dir = reverse ? -1 : 1;
    first = reverse ? up - 1 - row0 : row0;
  }
  __device__ __forceinline__ int row(int j) const { return first + dir * j; }
  // chunk c of the segment is the last one of a sweep forward in time
  __device__ __forceinline__ bool at_end(int c) const { return row0 + C * c + C >= len; }
};
// A head's rows of `width` elements of `es` bytes as a range-checked buffer.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, size_t head, int rows, int len, int width,
                                                            int es) {
  return make_rsrc((const unsigned char*)p + head * rows * width * es, (uint32_t)(len * width * es));
}
// The log decay of row j of a sweep: reversed row j carries that of the row after it (the first has none).
// As stored, in 32 bits; decay_of() widens it.
template <typename T>
__device__ __forceinline__ uint32_t load_decay(__amdgpu_buffer_rsrc_t gr, const Rows& R, int j, int reverse, int head_decay) {
  const int at = reverse ? R.up - j : j;
  const int off = (unsigned)at < (unsigned)R.len ? (head_decay ? 0 : at * (int)sizeof(T)) : 0x7FFFFFF0;   // out of range: 0
  if constexpr (sizeof(T) == 2) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(gr, off, 0, 0);
  else return __builtin_amdgcn_raw_buffer_load_b32(gr, off, 0, 0);
}
template <typename T>
__device__ __forceinline__ float decay_of(uint32_t w) {
  pin(w);   // not widened before: that would wait for the load
  return __uint_as_float(sizeof(T) == 2 ? w << 16 : w);
}
template <typename T>
__device__ __forceinline__ const T* decays_of(const SweepLaunch& L, int bh) {
  return (const T*)L.g + (L.head_decay ? (size_t)(bh % L.heads) : (size_t)bh * L.rows);
}
__device__ __forceinline__ void pin4(u32x4& x) { asm volatile("" : "+v"(x)); }

// N terms of wt z for the eight (four) elements of a piece, stored at p, p + stride, ..
template <typename T, int N>
__device__ __forceinline__ void store_scaled(unsigned char* p, int stride, Frag z, float wt) {
  if constexpr (sizeof(T) == 2) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = wt * ((e & 1) ? bf16_hi_half(z.w[e >> 1]) : bf16_lo_half(z.w[e >> 1]));
    Frag t[N];
    split_terms<N>(v, t);
#pragma unroll
    for (int n = 0; n < N; ++n) store_frag(p + n * stride, t[n]);
  } else {
    store_frag(p, frag_from_acc_f32(__builtin_bit_cast(f32x4, z.w) * wt));
  }
}
// A cell is one segment of one unit (key head of a batch entry); its parts
// (role, head of the group, slice) read the same rows of x and y.  Workgroups
// go to the 8 XCDs in turn, so the parts of a cell get ids equal modulo 8 and
// find each other's rows in their XCD's L2 -- where there are cells for every
// XCD; a few cells are spread over all of them instead.  (A whole
// unit in turn instead of a cell, with 4 units: every XCD read every key.)
constexpr int kXcds = 8;
__host__ __device__ inline bool cells_by_xcd(long long cells) { return cells % kXcds == 0 || cells >= 4 * kXcds; }
inline long long cell_workgroups(long long cells, int parts) {
  return (cells_by_xcd(cells) ? (cells + kXcds - 1) / kXcds * kXcds : cells) * parts;
}
// false: no cell (the ids are filled up to whole rounds of XCDs)
__device__ __forceinline__ bool cell_of(int cells, int parts, int& cell, int& part) {
  const int id = blockIdx.x;
  if (cells_by_xcd(cells)) {
    cell = (id / kXcds) / parts * kXcds + id % kXcds;
    part = (id / kXcds) % parts;
  } else {
    cell = id / parts;
    part = id % parts;
  }
  return cell < cells;
}

// Four consecutive elements of a row, as loaded.
template <typename T> struct Quad;
template <> struct Quad<bf16_t> {
  typedef u32x2 Raw;
  static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t b, int off) {
    return __builtin_amdgcn_raw_buffer_load_b64(b, off, 0, 0);
  }
  static __device__ __forceinline__ float get(Raw w, int j) {
    return (j & 1) ? bf16_hi_half(w[j >> 1]) : bf16_lo_half(w[j >> 1]);
  }
};
template <> struct Quad<float> {
  typedef f32x4 Raw;
  static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t b, int off) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
  }
  static __device__ __forceinline__ float get(Raw w, int j) { return w[j]; }
};

// EXACT: states with three bf16 terms (one is returned), else two.  PAD: roles
// of fewer than D1 state rows run among those of D1, with zeros in the rest.
template <typename T, int D1, int DS, bool EXACT, bool PAD>
__global__ __launch_bounds__(512, 2) void sweep_kernel(SweepLaunch L) {
  using S = SweepCfg<T, D1, DS, EXACT>;
  constexpr int E = S::E, KBN = S::KBN, KBC = S::KBC, NDV = S::NDV, TR = S::TR, TC = S::TC;
  constexpr bool BF = S::BF;
  __shared__ __attribute__((aligned(16))) unsigned char lds[S::LDS_BYTES];

  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const int g = lane / 16, r = lane % 16;
  int cell, part, role = 0;
  if (!cell_of(L.units * L.nseg, L.parts, cell, part)) return;
  const int unit = cell / L.nseg, seg = cell % L.nseg;
  while (role + 1 < L.nroles && part >= L.role[role].parts) part -= L.role[role++].parts;
  const SweepRole A = L.role[role];
  const int d1 = PAD ? A.d1 : D1;
  const int slices = A.d2 / DS;
  const int slice = part % slices;
  const int bh = unit * L.group + part / slices;
  const Rows R(L, bh, seg, L.seg_rows, A.reverse);
  const int len = R.len, nch = R.nch;
  auto dec_of = [&](int c) __attribute__((always_inline)) {
    return reinterpret_cast<float*>(lds + S::DEC_OFF + (c & 1) * S::DEC_BYTES);
  };
  unsigned char *ly = lds, *lz = lds + S::Z_OFF, *lzs = lds + S::ZS_OFF, *lh = lds + S::H_OFF;

  // Copies of Y, Z and the scaled Z to LDS, a chunk ahead in registers: units
  // y0 .. y1 - 1 of Y and z0 .. z1 - 1 of Z.  Loads and copies run on past the
  // last chunk (the last one again, into buffers nobody reads): a conditional
  // load would make every wait for an older one wait for all loads in flight.
  const __amdgpu_buffer_rsrc_t yr = rows_rsrc(A.y, A.y_shared ? unit : bh, L.rows, len, d1, E);
  const __amdgpu_buffer_rsrc_t zr = rows_rsrc(A.z, A.z_shared ? unit : bh, L.rows, len, A.d2, E);
  const int ct = tid & 255;
  const bool ypad = PAD && ct % S::YPR * 16 >= d1 * E;   // (256 threads are whole rows of pieces)
  constexpr int YM = S::NY - S::YO, ZM = S::NZ - S::ZO;   // (the state waves have the most)
  struct Units {
    Frag y[YM], z[ZM];
  };
  auto load = [&](Units& u, int c, auto state) __attribute__((always_inline)) {
    constexpr bool ST = decltype(state)::value;
    constexpr int y0 = ST ? S::YO : 0, ny = ST ? YM : S::YO, z0 = ST ? S::ZO : 0, nz = ST ? ZM : S::ZO;
#pragma unroll
    for (int j = 0; j < ny; ++j) {
      const int p = ct + 256 * (y0 + j);
      const int off = R.row(C * c + p / S::YPR) * d1 * E + (p % S::YPR) * 16;
      u.y[j].w = __builtin_amdgcn_raw_buffer_load_b128(yr, ypad ? 0x7FFFFFF0 : off, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < nz; ++j) {
      const int p = ct + 256 * (z0 + j);
      u.z[j].w = __builtin_amdgcn_raw_buffer_load_b128(
          zr, (R.row(C * c + p / S::ZPR) * A.d2 + slice * DS) * E + (p % S::ZPR) * 16, 0, 0);
    }
  };
  auto place = [&](Units& u, int c, auto state) __attribute__((always_inline)) {
    constexpr bool ST = decltype(state)::value;
    constexpr int y0 = ST ? S::YO : 0, ny = ST ? YM : S::YO, z0 = ST ? S::ZO : 0, nz = ST ? ZM : S::ZO;
    const float* dec = dec_of(c);
    // the copies' uses of the loads are tied to here: moved up into an earlier
    // phase they would make it wait for them
#pragma unroll
    for (int j = 0; j < ny; ++j) pin4(u.y[j].w);
#pragma unroll
    for (int j = 0; j < nz; ++j) pin4(u.z[j].w);
    // (read before anything is written: a wait for them then waits for no write)
    float wt[nz > 0 ? nz : 1];   // G(C, row)
#pragma unroll
    for (int j = 0; j < nz; ++j) wt[j] = dec[3 * C + min(ct + 256 * (z0 + j), C * S::ZPR - 1) / S::ZPR];
#pragma unroll
    for (int j = 0; j < ny; ++j) {
      const int p = ct + 256 * (y0 + j);
      if (C * S::YPR % 256 == 0 || p < C * S::YPR) store_frag(ly + lds_piece<S::YROW>(p / S::YPR, p % S::YPR), u.y[j]);
    }
#pragma unroll
    for (int j = 0; j < nz; ++j) {
      const int p = ct + 256 * (z0 + j);
      if (C * S::ZPR % 256 == 0 || p < C * S::ZPR) {
        const int off = lds_piece<S::ZROW>(p / S::ZPR, p % S::ZPR);
        store_frag(lz + off, u.z[j]);
        store_scaled<T, S::ZSETS>(lzs + off, S::Z_BYTES, u.z[j], wt[j]);
      }
    }
  };

  if (wave < 4) {
    // ============================================================ output waves
    const __amdgpu_buffer_rsrc_t xr = rows_rsrc(A.x, A.x_shared ? unit : bh, L.rows, len, d1, E);
    const __amdgpu_buffer_rsrc_t outr = rows_rsrc(A.out, bh, L.rows, len, A.d2, A.out_f32 ? 4 : E);
    const __amdgpu_buffer_rsrc_t wr = rows_rsrc(A.w, A.w_shared ? unit : bh, L.rows, len, A.d2, A.w ? E : 0);
    const int t = 16 * wave + r;      // this lane's row of the chunk
    const RowFrags<S::YROW, KBN, false> yrow(0, g, r);
    const RowFrags<S::YROW, KBN, true> hrow(S::H_OFF, g, r);
    ColFrags<T, S::ZROW> zcol[NDV];
#pragma unroll
    for (int d = 0; d < NDV; ++d) zcol[d].set(S::Z_OFF, 16 * d, g, r);
    Frag xf[KBN];                     // this lane's row of X
    auto load_x = [&](int c) __attribute__((always_inline)) {
      const int row = R.row(C * c + t);
#pragma unroll
      for (int kb = 0; kb < KBN; ++kb) {
        const int off = row * d1 * E + kb * 64 + g * 16;
        const bool pad = (PAD || D1 < S::KB) && kb * 64 + g * 16 >= d1 * E;
        xf[kb].w = __builtin_amdgcn_raw_buffer_load_b128(xr, pad ? 0x7FFFFFF0 : off, 0, 0);
      }
    };
    constexpr std::false_type OUTPUT{};
    Units u0;
    load(u0, 0, OUTPUT);
    load_x(0);
    lds_barrier();   // the first decay factors are there
    place(u0, 0, OUTPUT);
    load(u0, min(1, R.last), OUTPUT);
    lds_barrier();   // the first operands are there
    // One copy of the loop per wave: W, the wave's row tile, fixes how many
    // tiles of P it has, and DOT whether it forms the dots, so that the body is
    // straight-line code and every wait counts the loads in flight exactly.
    auto run = [&](auto wconst, auto dotconst) __attribute__((always_inline)) {
      constexpr int W = decltype(wconst)::value;
      constexpr bool DOT = decltype(dotconst)::value;
      constexpr int NPB = (16 * W) / S::KB + 1;      // K blocks of P^T it multiplies
      for (int c = 0; c < nch; ++c) {
        const float* dec = dec_of(c);
        const int row = R.row(C * c + t);
        typename Quad<T>::Raw wv[NDV];   // four elements of w each
        if constexpr (DOT) {
#pragma unroll
          for (int d = 0; d < NDV; ++d) wv[d] = Quad<T>::load(wr, (row * A.d2 + slice * DS + 16 * d + 4 * g) * E);
        }
        // ---- phase 1: H^T X^T, and the tiles of Y X^T up to this wave's own
        f32x4 oacc[NDV], p[RT];
#pragma unroll
        for (int d = 0; d < NDV; ++d) oacc[d] = zero4();
#pragma unroll
        for (int i = 0; i < RT; ++i) p[i] = zero4();
        // Operand fragments are read one step ahead of the products that take
        // them; a step is one K block of up to four state column tiles, or of
        // the tiles of Y.
        constexpr int DG = NDV < 4 ? NDV : 4, NG = NDV / DG;
        constexpr int NF = S::HSETS * DG > W + 1 ? S::HSETS * DG : W + 1;
        Frag f[2][NF];
        auto read = [&](int step) __attribute__((always_inline)) {
          Frag* to = f[step & 1];
          const int kb = step / (NG + 1), grp = step % (NG + 1);
          if (grp < NG) {
#pragma unroll
            for (int i = 0; i < S::HSETS * DG; ++i)
              to[i] = hrow.read(lds, grp * DG + i % DG, kb, (i / DG) * S::H_BYTES);
          } else {
#pragma unroll
            for (int i = 0; i <= W; ++i) to[i] = yrow.read(lds, i, kb);
          }
        };
        read(0);
#pragma unroll
        for (int step = 0; step < KBN * (NG + 1); ++step) {
          if (step + 1 < KBN * (NG + 1)) read(step + 1);
          __builtin_amdgcn_sched_barrier(0);
          const Frag* from = f[step & 1];
          const int kb = step / (NG + 1), grp = step % (NG + 1);
          if (grp < NG) {
#pragma unroll
            for (int i = S::HSETS * DG - 1; i >= 0; --i) {
              f32x4& o = oacc[grp * DG + i % DG];
              o = mma<T>(o, from[i], xf[kb]);
            }
          } else {
#pragma unroll
            for (int i = 0; i <= W; ++i) p[i] = mma<T>(p[i], from[i], xf[kb]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        Frag zf[NPB][NDV];
#pragma unroll
        for (int kb = 0; kb < NPB; ++kb)
#pragma unroll
          for (int d = 0; d < NDV; ++d) zf[kb][d] = zcol[d].read(lds, kb);
        load_x(min(c + 1, R.last));
        lds_barrier();
        // ---- phase 2: P^T = G . (Y X^T).  Below the diagonal G(t, s) is
        // G(t, e) G(e, s) with e the last row of the tile of s: both at most 1
        // for decays, one exponential a tile here and one a row of the chunk
        // (decay_factors).
        const float ch = dec[t], cl = dec[C + t];
        f32x4 self = zero4();   // with dots: the row's pair with itself, which is not part of them
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float rowf = __builtin_amdgcn_exp2f((ch - dec[16 * i + 15]) + (cl - dec[C + 16 * i + 15]));
          const f32x4 tail = *reinterpret_cast<const f32x4*>(dec + 4 * C + 16 * i + 4 * g);
          p[i] *= tail * rowf;
        }
        {
          const f32x4 sh = *reinterpret_cast<const f32x4*>(dec + 16 * W + 4 * g);
          const f32x4 sl = *reinterpret_cast<const f32x4*>(dec + C + 16 * W + 4 * g);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = p[W][j] * __builtin_amdgcn_exp2f((ch - sh[j]) + (cl - sl[j]));
            p[W][j] = (DOT ? 4 * g + j < r : 4 * g + j <= r) ? x : 0.f;
            if constexpr (DOT) self[j] = 4 * g + j == r ? x : 0.f;
          }
        }
        const float gam = dec[2 * C + t];
#pragma unroll
        for (int d = 0; d < NDV; ++d) oacc[d] *= gam;
        // this slice's part of w_t . out_t, of what the accumulators hold
        auto dot = [&]() __attribute__((always_inline)) {
          float x = 0.f;
#pragma unroll
          for (int d = 0; d < NDV; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) x = __builtin_fmaf(Quad<T>::get(wv[d], j), oacc[d][j], x);
          return x;   // this lane's columns
        };
        float before = 0.f;   // of the rows before the chunk
        if constexpr (DOT) {
#pragma unroll
          for (int d = 0; d < NDV; ++d) pin(wv[d]);
          before = dot();
        }
        // O^T += Z^T P^T
#pragma unroll
        for (int kb = 0; kb < NPB; ++kb) {
          Frag ph, pl;
          if constexpr (BF) {
            const f32x4 u = p[2 * kb], v = p[2 * kb + 1];
            const float w[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
            Frag two[2];
            split_terms<2>(w, two);
            ph = two[0], pl = two[1];
          }
          else ph = frag_from_acc_f32(p[kb]);
#pragma unroll
          for (int d = 0; d < NDV; ++d) {
            if constexpr (BF) oacc[d] = mma<T>(oacc[d], zf[kb][d], pl);
            oacc[d] = mma<T>(oacc[d], zf[kb][d], ph);
          }
        }
        if constexpr (DOT) {
          const float both = dot();
          // (bf16: both terms in one product, the tile's rows of Z in both halves of the K block)
          Frag f;
          if constexpr (BF) {
            uint32_t ha, la, hb, lb;
            split2(self[0], self[1], ha, la);
            split2(self[2], self[3], hb, lb);
            f.w = u32x4{ha, hb, la, lb};
          } else f = frag_from_acc_f32(self);
#pragma unroll
          for (int d = 0; d < NDV; ++d) {
            const u32x4 z = zf[NPB - 1][d].w;
            constexpr int at = W & 1 ? 2 : 0;
            oacc[d] = mma<T>(oacc[d], BF ? Frag{u32x4{z[at], z[at + 1], z[at], z[at + 1]}} : zf[NPB - 1][d], f);
          }
          const float in = row_groups_sum(both - before);
          before = row_groups_sum(before);
          if (g == 0 && (unsigned)row < (unsigned)len) {
            float* to = A.dot + ((size_t)slice * L.units * L.group + bh) * L.rows + row;
            to[0] = before;
            to[(size_t)slices * L.units * L.group * L.rows] = in;
          }
        }
        // this lane holds four consecutive columns of row t
#pragma unroll
        for (int d = 0; d < NDV; ++d) {
          const int col = slice * DS + 16 * d + 4 * g;
          if (A.out_f32) store4<float>(outr, (row * A.d2 + col) * 4, oacc[d]);
          else store4<T>(outr, (row * A.d2 + col) * E, oacc[d]);
        }
        place(u0, c + 1, OUTPUT);
        load(u0, min(c + 2, R.last), OUTPUT);
        lds_barrier();
      }
    };
    auto run_wave = [&](auto dotconst) __attribute__((always_inline)) {
      switch (wave) {
        case 0: run(std::integral_constant<int, 0>{}, dotconst); break;
        case 1: run(std::integral_constant<int, 1>{}, dotconst); break;
        case 2: run(std::integral_constant<int, 2>{}, dotconst); break;
        default: run(std::integral_constant<int, 3>{}, dotconst); break;
      }
    };
    if (A.w) run_wave(std::true_type{});
    else run_wave(std::false_type{});
  } else {
    // ============================================================ state waves
    const int sw = wave - 4;
    const int ct0 = (sw % S::WC) * TC, rt0 = (sw / S::WC) * TR;   // this wave's first column and row tile
    const T* gp = decays_of<T>(L, bh);
    const __amdgpu_buffer_rsrc_t gr = make_rsrc(gp, (uint32_t)((L.head_decay ? 1 : len) * E));
    uint32_t gv;   // the next chunk's log decay of row `lane`
    auto load_g = [&](int c) __attribute__((always_inline)) {
      gv = load_decay<T>(gr, R, R.row0 + C * c + lane, A.reverse, L.head_decay);
    };
    ColFrags<T, S::YROW> ycol[TR];
    ColFrags<T, S::ZROW> zcol[TC];
#pragma unroll
    for (int i = 0; i < TR; ++i) ycol[i].set(0, 16 * min(rt0 + i, S::RH - 1), g, r);
#pragma unroll
    for (int j = 0; j < TC; ++j) zcol[j].set(S::ZS_OFF, 16 * (ct0 + j), g, r);
    // the state slice: lane (g, r) holds rows 4 g .. 4 g + 3 of column r of each of its tiles
    f32x4 h[TR][TC];
    const size_t sbase = (size_t)bh * d1 * A.d2;
    auto state_at = [&](int i, int j, int e) __attribute__((always_inline)) {   // element offset inside one head's state
      const int row = 16 * (rt0 + i) + 4 * g + e, col = slice * DS + 16 * (ct0 + j) + r;
      return A.turned ? col * d1 + row : row * A.d2 + col;
    };
    auto own = [&](int i) __attribute__((always_inline)) { return S::WR * TR == S::RH || rt0 + i < S::RH; };
    auto stored = [&](int i) __attribute__((always_inline)) { return own(i) && (!PAD || 16 * (rt0 + i) < d1); };
    const float* init = L.nseg > 1 ? A.seg_states + (size_t)seg * L.seg_subs * L.seg_stride : A.init;
#pragma unroll
    for (int i = 0; i < TR; ++i)
#pragma unroll
      for (int j = 0; j < TC; ++j) {
        h[i][j] = zero4();
        if (init && stored(i)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) h[i][j][e] = init[sbase + state_at(i, j, e)];
        }
      }
    int hput[TR];   // offsets of this lane's rows of H^T, by row tile
#pragma unroll
    for (int i = 0; i < TR; ++i) {
      hput[i] = S::H_OFF + (BF ? state_piece<S::YROW>(16 * ct0 + r, 2 * (rt0 + i) + (g >> 1)) + (g & 1) * 8
                               : state_piece<S::YROW>(16 * ct0 + r, 4 * (rt0 + i) + g));
      asm("" : "+v"(hput[i]));
    }
    auto put_state = [&]() __attribute__((always_inline)) {   // H^T [column][row] as the A operand of H^T X^T
#pragma unroll
      for (int i = 0; i < TR; ++i)
#pragma unroll
        for (int j = 0; j < TC; ++j) {
          if (!own(i)) continue;
          const f32x4 x = h[i][j];
          if constexpr (BF) {
            unsigned char* to = lds + hput[i] + j * 16 * S::YROW;
            uint32_t ha, la, hb, lb;
            split2(x[0], x[1], ha, la);
            split2(x[2], x[3], hb, lb);
            *reinterpret_cast<u32x2*>(to) = u32x2{ha, hb};
            *reinterpret_cast<u32x2*>(to + S::H_BYTES) = u32x2{la, lb};
          } else {
            *reinterpret_cast<f32x4*>(lds + hput[i] + j * 16 * S::YROW) = x;
          }
        }
    };
    constexpr std::true_type STATE{};
    Units u0, u1;   // of even chunks and of odd ones (NR == 1: u0 of all)
    load_g(0);
    load(u0, 0, STATE);
    if constexpr (S::NR == 2) load(u1, min(1, R.last), STATE);
    if constexpr (S::D1P != D1) {
      // half K blocks: the columns behind D1 are zero for good
      for (int p = tid - 256; p < 2 * (C > DS ? C : DS); p += 256) {
        const int row = p >> 1, piece = 2 + (p & 1);
        if (row < C) store_frag(ly + lds_piece<S::YROW>(row, piece), Frag{u32x4{0, 0, 0, 0}});
        if (row < DS) {
          store_frag(lh + state_piece<S::YROW>(row, piece), Frag{u32x4{0, 0, 0, 0}});
          store_frag(lh + S::H_BYTES + state_piece<S::YROW>(row, piece), Frag{u32x4{0, 0, 0, 0}});
        }
      }
    }
    if (sw == 0) decay_factors(decay_of<T>(gv), dec_of(0), lane, A.drop_end && R.at_end(0));
    put_state();
    lds_barrier();   // the first decay factors are there
    place(u0, 0, STATE);
    load_g(min(1, R.last));
    load(u0, min(S::NR, R.last), STATE);
    lds_barrier();   // the first operands are there
    auto chunk = [&](int c, Units& next) __attribute__((always_inline)) {
      // ---- phase 1.  A operand: the columns of Y this wave's row tiles are;
      // B operand: the terms of G(C, s) z_s for its column tile
      const float end = dec_of(c)[2 * C + C - 1], less = dec_of(c)[kDecSets * C];
      if (sw == 0) decay_factors(decay_of<T>(gv), dec_of(c + 1), lane, A.drop_end && R.at_end(c + 1));
      decay_step<TR, TC>(h, end, less);
      // fp32: the chunk's products are summed apart and added to the state once;
      // on top of it each of the 16 would round at the state's size (bf16: two,
      // for which there are no registers in the widest slices)
      f32x4 sum[BF ? 1 : TR][BF ? 1 : TC];
      if constexpr (!BF) {
#pragma unroll
        for (int i = 0; i < TR; ++i)
#pragma unroll
          for (int j = 0; j < TC; ++j) sum[i][j] = zero4();
      }
      constexpr int KA = BF ? KBC : 1;   // K blocks read ahead of the products (fp32: one, for the registers)
      Frag zf[KA][TC][S::ZSETS], yf[KA][TR];
      auto read = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TR; ++i) yf[kb % KA][i] = ycol[i].read(lds, kb);
#pragma unroll
        for (int j = 0; j < TC; ++j)
#pragma unroll
          for (int n = 0; n < S::ZSETS; ++n) zf[kb % KA][j][n] = zcol[j].read(lds, kb, n * S::Z_BYTES);
      };
      auto multiply = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int n = S::ZSETS - 1; n >= 0; --n)
#pragma unroll
          for (int j = 0; j < TC; ++j)
#pragma unroll
            for (int i = 0; i < TR; ++i) {
              f32x4& to = BF ? h[i][j] : sum[BF ? 0 : i][BF ? 0 : j];
              to = mma<T>(to, yf[kb % KA][i], zf[kb % KA][j][n]);
            }
      };
#pragma unroll
      for (int kb = 0; kb < KA; ++kb) read(kb);
#pragma unroll
      for (int kb = KA; kb < KBC; ++kb) {
        multiply(kb - KA);
        read(kb);
      }
#pragma unroll
      for (int kb = KBC - KA; kb < KBC; ++kb) multiply(kb);
      if constexpr (!BF) {
#pragma unroll
        for (int i = 0; i < TR; ++i)
#pragma unroll
          for (int j = 0; j < TC; ++j) h[i][j] += sum[i][j];
      }
      lds_barrier();
      // ---- phase 2
      place(next, c + 1, STATE);
      load_g(min(c + 2, R.last));
      load(next, min(c + 1 + S::NR, R.last), STATE);
      put_state();
      lds_barrier();
    };
    for (int c = 0; c < nch; c += 2) {
      chunk(c, S::NR == 2 ? u1 : u0);
      if (c + 1 >= nch) break;
      chunk(c + 1, u0);
    }
    // the final state, of the last segment
    if (A.fin && seg == L.nseg - 1) {
      // dh0 = a_1 R_1: the first row's own decay, which a reversed sweep has not applied
      float scale = 1.f;
      if (A.reverse && len > 0) {
        const float x = to_f32(*gp) * kLog2E;
        scale = __builtin_amdgcn_exp2f(x < kDecayFloor ? kDecayFloor : x);
      }
#pragma unroll
      for (int i = 0; i < TR; ++i)
#pragma unroll
        for (int j = 0; j < TC; ++j) {
          if (!stored(i)) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) A.fin[sbase + state_at(i, j, e)] = h[i][j][e] * scale;
        }
    }
  }
}

// A segment's own state, from zero: sum_s G(end, s) y_s z_s^T, and its whole
// decay.  One workgroup holds the whole [D1, D2] state of one (batch, head) in
// the accumulators of its eight waves (two rows of waves, four columns), so
// that every row of Y and Z is read once; per chunk it copies Y and the terms
// of the scaled Z to LDS and multiplies Y^T (G(C, .) Z), in two phases with a
// barrier each as above.  Two workgroups a CU.  B1 H16 Hk4 T32768 d128, bf16:
// 66 us, 2.4 TB/s: bound by the latency of a chunk's loads, its two barriers
// and the forming of the terms; the products are a third of it.
template <typename T, int D1, int D2>
struct OwnCfg {
  static constexpr int E = (int)sizeof(T);
  static constexpr int KBC = C / FragTraits<T>::KB;
  static constexpr int YROW = D1 * E < 32 ? 32 : D1 * E, ZROW = D2 * E < 32 ? 32 : D2 * E;
  static constexpr int ZSETS = E == 2 ? 3 : 1;
  static constexpr int RH = D1 / 16, RD = D2 / 16;
  static constexpr int TR = (RH + 1) / 2, TC = (RD + 3) / 4;   // tiles of one wave
  static constexpr int Y_BYTES = C * YROW, Z_BYTES = C * ZROW;
  static constexpr int DEC_OFF = Y_BYTES + ZSETS * Z_BYTES, DEC_BYTES = kDecFloats * 4;
  static constexpr int LDS_BYTES = DEC_OFF + 2 * DEC_BYTES;
  static constexpr int YPR = D1 * E / 16, ZPR = D2 * E / 16;
  static constexpr int NY = (C * YPR + 511) / 512, NZ = (C * ZPR + 511) / 512;
};

template <typename T, int D1, int D2>
__global__ __launch_bounds__(512, sizeof(T) == 2 ? 4 : 2) void own_state_kernel(SweepLaunch L) {
  using S = OwnCfg<T, D1, D2>;
  constexpr int E = S::E;
  __shared__ __attribute__((aligned(16))) unsigned char lds[S::LDS_BYTES];
  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const int g = lane / 16, r = lane % 16;
  int cell, part;
  if (!cell_of(L.units * L.nseg, L.parts, cell, part)) return;
  const int unit = cell / L.nseg, seg = cell % L.nseg;
  const SweepRole A = L.role[part / L.group];   // (a direction)
  const int bh = unit * L.group + part % L.group;
  const Rows R(L, bh, seg, L.seg_rows, A.reverse);
  auto dec_of = [&](int c) __attribute__((always_inline)) {
    return reinterpret_cast<float*>(lds + S::DEC_OFF + (c & 1) * S::DEC_BYTES);
  };
  unsigned char *ly = lds, *lzs = lds + S::Y_BYTES;
  const __amdgpu_buffer_rsrc_t yr = rows_rsrc(A.y, A.y_shared ? unit : bh, L.rows, R.len, D1, E);
  const __amdgpu_buffer_rsrc_t zr = rows_rsrc(A.z, A.z_shared ? unit : bh, L.rows, R.len, D2, E);
  const __amdgpu_buffer_rsrc_t gr = make_rsrc(decays_of<T>(L, bh), (uint32_t)((L.head_decay ? 1 : R.len) * E));
  Frag yv[S::NY], zv[S::NZ];
  uint32_t gv;
  auto load = [&](int c) __attribute__((always_inline)) {
    gv = load_decay<T>(gr, R, R.row0 + C * c + lane, A.reverse, L.head_decay);
#pragma unroll
    for (int j = 0; j < S::NY; ++j) {
      const int p = tid + 512 * j;
      yv[j].w = __builtin_amdgcn_raw_buffer_load_b128(yr, R.row(C * c + p / S::YPR) * D1 * E + (p % S::YPR) * 16, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < S::NZ; ++j) {
      const int p = tid + 512 * j;
      zv[j].w = __builtin_amdgcn_raw_buffer_load_b128(zr, R.row(C * c + p / S::ZPR) * D2 * E + (p % S::ZPR) * 16, 0, 0);
    }
  };
  auto place = [&](int c) __attribute__((always_inline)) {
    const float* dec = dec_of(c);
#pragma unroll
    for (int j = 0; j < S::NY; ++j) pin4(yv[j].w);
#pragma unroll
    for (int j = 0; j < S::NZ; ++j) pin4(zv[j].w);
    float wt[S::NZ];
#pragma unroll
    for (int j = 0; j < S::NZ; ++j) wt[j] = dec[3 * C + min(tid + 512 * j, C * S::ZPR - 1) / S::ZPR];
#pragma unroll
    for (int j = 0; j < S::NY; ++j) {
      const int p = tid + 512 * j;
      if (C * S::YPR % 512 == 0 || p < C * S::YPR) store_frag(ly + lds_piece<S::YROW>(p / S::YPR, p % S::YPR), yv[j]);
    }
#pragma unroll
    for (int j = 0; j < S::NZ; ++j) {
      const int p = tid + 512 * j;
      if (C * S::ZPR % 512 == 0 || p < C * S::ZPR)
        store_scaled<T, S::ZSETS>(lzs + lds_piece<S::ZROW>(p / S::ZPR, p % S::ZPR), S::Z_BYTES, zv[j], wt[j]);
    }
  };
  const int rt0 = (wave / 4) * S::TR, ct0 = (wave % 4) * S::TC;
  auto rt = [&](int i) __attribute__((always_inline)) { return min(rt0 + i, S::RH - 1); };   // (spare waves repeat the last tile)
  auto ctl = [&](int j) __attribute__((always_inline)) { return min(ct0 + j, S::RD - 1); };
  ColFrags<T, S::YROW> ycol[S::TR];
  ColFrags<T, S::ZROW> zcol[S::TC];
#pragma unroll
  for (int i = 0; i < S::TR; ++i) ycol[i].set(0, 16 * rt(i), g, r);
#pragma unroll
  for (int j = 0; j < S::TC; ++j) zcol[j].set(S::Y_BYTES, 16 * ctl(j), g, r);
  f32x4 h[S::TR][S::TC];
#pragma unroll
  for (int i = 0; i < S::TR; ++i)
#pragma unroll
    for (int j = 0; j < S::TC; ++j) h[i][j] = zero4();
  load(0);
  if (wave == 0) decay_factors(decay_of<T>(gv), dec_of(0), lane, A.drop_end && R.at_end(0));
  lds_barrier();
  place(0);
  load(min(1, R.last));
  lds_barrier();
  float log_h = 0.f, log_l = 0.f;   // the segment's log2 decay, whole part and rest
  for (int c = 0; c < R.nch; ++c) {
    if (wave == 0) decay_factors(decay_of<T>(gv), dec_of(c + 1), lane, A.drop_end && R.at_end(c + 1));
    const float end = dec_of(c)[2 * C + C - 1], less = dec_of(c)[kDecSets * C];
    log_h += dec_of(c)[C - 1];
    log_l += dec_of(c)[2 * C - 1];
    decay_step<S::TR, S::TC>(h, end, less);
    constexpr bool APART = E == 4;   // (as in sweep_kernel)
    f32x4 sum[APART ? S::TR : 1][APART ? S::TC : 1];
    if constexpr (APART) {
#pragma unroll
      for (int i = 0; i < S::TR; ++i)
#pragma unroll
        for (int j = 0; j < S::TC; ++j) sum[i][j] = zero4();
    }
#pragma unroll
    for (int kb = 0; kb < S::KBC; ++kb) {
      Frag yf[S::TR];
#pragma unroll
      for (int i = 0; i < S::TR; ++i) yf[i] = ycol[i].read(lds, kb);
#pragma unroll
      for (int n = S::ZSETS - 1; n >= 0; --n)
#pragma unroll
        for (int j = 0; j < S::TC; ++j) {
          const Frag zf = zcol[j].read(lds, kb, n * S::Z_BYTES);
#pragma unroll
          for (int i = 0; i < S::TR; ++i) {
            f32x4& to = APART ? sum[APART ? i : 0][APART ? j : 0] : h[i][j];
            to = mma<T>(to, yf[i], zf);
          }
        }
    }
    if constexpr (APART) {
#pragma unroll
      for (int i = 0; i < S::TR; ++i)
#pragma unroll
        for (int j = 0; j < S::TC; ++j) h[i][j] += sum[i][j];
    }
    lds_barrier();
    place(c + 1);
    load(min(c + 2, R.last));
    lds_barrier();
  }
  float* out = A.seg_out + (size_t)seg * L.seg_stride + (size_t)bh * D1 * D2;
#pragma unroll
  for (int i = 0; i < S::TR; ++i)
#pragma unroll
    for (int j = 0; j < S::TC; ++j)
      if (rt0 + i < S::RH && ct0 + j < S::RD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[(16 * (rt0 + i) + 4 * g + e) * D2 + 16 * (ct0 + j) + r] = h[i][j][e];
      }
  if (tid == 0) {
    const float x = log_h + log_l;
    A.seg_decay[(size_t)seg * L.units * L.group + bh] = float2{__builtin_amdgcn_exp2f(x), decay_less_one(x)};
  }
}

// Segment states, in place: segment i holds its own state (from zero) on entry
// and its start on return, start[0] = init, start[i + 1] = decay_i start[i] +
// own_i.  One thread per four state elements of one (batch, head); the
// workgroups' second plane is the backward's second direction.  HBM-bound, with
// AHEAD segments' loads in flight: 11 us for the 64 MB of 16 heads, 32
// sub-segments, d128.
struct ScanArgs {
  float* states;
  const float2* decay;   // of every segment, and less 1 (as decay_step takes them)
  const float* init;
};
__global__ __launch_bounds__(256) void segment_scan_kernel(ScanArgs one, ScanArgs two, int nseg, int heads,
                                                           long long elems, long long seg_stride) {
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= heads * elems) return;
  float* states = blockIdx.y ? two.states : one.states;
  const float2* decay = blockIdx.y ? two.decay : one.decay;
  const float* init = blockIdx.y ? two.init : one.init;
  const int bh = (int)(i / elems);
  f32x4 h = init ? *reinterpret_cast<const f32x4*>(init + i) : zero4();
  constexpr int AHEAD = 8;   // segments whose loads are in flight together
  for (int s0 = 0; s0 < nseg; s0 += AHEAD) {
    f32x4 mine[AHEAD];
    float2 d[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int s = min(s0 + j, nseg - 2);   // (the last segment's own state is not formed)
      mine[j] = *reinterpret_cast<const f32x4*>(states + s * seg_stride + i);
      d[j] = decay[(size_t)s * heads + bh];
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (s0 + j >= nseg) break;
      *reinterpret_cast<f32x4*>(states + (s0 + j) * seg_stride + i) = h;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        h[e] = (d[j].y != 0.f ? __builtin_fmaf(h[e], d[j].y, h[e]) : d[j].x * h[e]) + mine[j][e];
    }
  }
}

template <typename T, int D1, int DS, bool EXACT, bool PAD>
hipError_t launch_sweep_t(const SweepLaunch& L, hipStream_t stream) {
  const long long wgs = cell_workgroups((long long)L.units * L.nseg, L.parts);
  if (wgs == 0) return hipSuccess;
  hipLaunchKernelGGL((sweep_kernel<T, D1, DS, EXACT, PAD>), dim3((unsigned)wgs), dim3(512), 0, stream, L);
  return hipGetLastError();
}

constexpr int kPadSlice = 32;   // widest slices of launches that pad roles
template <typename T, int D1, int DS, bool PAD>
hipError_t launch_sweep_p(const SweepLaunch& L, hipStream_t stream) {
  constexpr bool F = sizeof(T) == 4;   // fp32 states have one term: one instantiation
  return L.exact_state || F ? launch_sweep_t<T, D1, DS, true, PAD>(L, stream) : launch_sweep_t<T, D1, DS, F, PAD>(L, stream);
}
template <typename T, int D1, int DS>
hipError_t launch_sweep_x(const SweepLaunch& L, hipStream_t stream) {
  for (int i = 0; i < L.nroles; ++i)
    if (L.role[i].d1 != D1) {
      if constexpr (DS <= kPadSlice && D1 > 16) return launch_sweep_p<T, D1, DS, true>(L, stream);
      else return hipErrorInvalidValue;
    }
  return launch_sweep_p<T, D1, DS, false>(L, stream);
}

template <typename T, int D1>
hipError_t launch_sweep_d(const SweepLaunch& L, int ds, hipStream_t stream) {
  switch (ds) {
    case 16: return launch_sweep_x<T, D1, 16>(L, stream);
    case 32: return launch_sweep_x<T, D1, 32>(L, stream);
    case 64: return launch_sweep_x<T, D1, 64>(L, stream);
    case 128:
      if constexpr (sizeof(T) == 2) return launch_sweep_x<T, D1, 128>(L, stream);
      break;
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_sweep_e(const SweepLaunch& L, int d1, int ds, hipStream_t stream) {
  switch (d1) {
    case 16: return launch_sweep_d<T, 16>(L, ds, stream);
    case 32: return launch_sweep_d<T, 32>(L, ds, stream);
    case 64: return launch_sweep_d<T, 64>(L, ds, stream);
    case 128: return launch_sweep_d<T, 128>(L, ds, stream);
  }
  return hipErrorInvalidValue;
}

template <typename T, int D1, int D2>
hipError_t launch_own_t(const SweepLaunch& L, hipStream_t stream) {
  const long long wgs = cell_workgroups((long long)L.units * L.nseg, L.parts);
  if (wgs == 0) return hipSuccess;
  hipLaunchKernelGGL((own_state_kernel<T, D1, D2>), dim3((unsigned)wgs), dim3(512), 0, stream, L);
  return hipGetLastError();
}

template <typename T, int D1>
hipError_t launch_own_d(const SweepLaunch& L, hipStream_t stream) {
  switch (L.role[0].d2) {
    case 16: return launch_own_t<T, D1, 16>(L, stream);
    case 32: return launch_own_t<T, D1, 32>(L, stream);
    case 64: return launch_own_t<T, D1, 64>(L, stream);
    case 128: return launch_own_t<T, D1, 128>(L, stream);
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_own_e(const SweepLaunch& L, int d1, hipStream_t stream) {
  switch (d1) {
    case 16: return launch_own_d<T, 16>(L, stream);
    case 32: return launch_own_d<T, 32>(L, stream);
    case 64: return launch_own_d<T, 64>(L, stream);
    case 128: return launch_own_d<T, 128>(L, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// ---------------------------------------------------------------- decay gradient
// dg_t = a_t <R_t, H_{t-1}> is everything that passes gate t: the pairs of a
// key s before t and a query u from t on, with the initial state among the keys
// and dhT among the queries.  The dots q_u . dq_u (every pair ending at u) less
// k_s . dk_s (every pair starting at s), summed over all rows from t on, give
// it too, but with the rounding errors of the largest pairs anywhere behind t:
// of strong decays nothing is left.  So pairs that pass no gate (a token with
// itself, the last token with dhT) are never added, and the sum is taken chunk
// by chunk.  For t in chunk c, rows u and s of that chunk only:
//   dg_t = sum_{u >= t} (i_u - j_u) + sum_{u >= t} a_u + sum_{s < t} b_s + X_c
// with q_u . dq_u = a_u (keys before the chunk) + i_u (in it, before u) and
// k_s . dk_s = b_s (queries after the chunk) + j_s (in it, after s), which the
// sweeps leave per slice from their unrounded outputs; X_c is what passes the
// whole chunk.  Of the last chunk that is <dhT, H> with H its start state,
// decayed; of the others a running sum again, but over chunks,
//   X_c = X_{c+1} + sum_{u in c+1} a_u - sum_{s in c} b_s,
// which starts anew, from 0, where the chunk lets less than 2^-16 pass and the
// sum is not above its own rounding error: 2^-19 (fp32 inputs: 2^-23) of the sum
// of |a| and |b| of one of the two chunks, the dots of bf16 inputs coming from
// states and pairs of 16 bits.  A decay factor below 2^-126 counts as 0: dg_t is
// 0 there, and no sum crosses it.
// What is left: dg_t is off by some 2^-18 (2^-22) of the pairs that pass any gate
// of its own chunk or the next.  A single gate much
// stronger than those around it, with a gradient that much smaller than theirs,
// keeps fewer digits of its own.
//
// One workgroup per (batch, head); a wave has CPW of the 16 CPW chunks of a
// round, from the sequence's end, a lane a row: the sums inside a chunk are
// fp32 prefix sums of the wave; one wave runs X over the round's chunks, in
// fp64, as are the sums of dhT and of a constant decay.  Of the latter, whose
// gradient is the sum over rows and batch, each workgroup leaves its sum for a
// second kernel, but for a single batch entry.  (One workgroup per head over the
// batch entries in turn saves that launch of some 2 us, and loses from two
// entries on.)
// Bound by the latency of its loads, scans and barriers: 8.4 us for the one slice
// of B4 H16 T4096, 6.5 for the four of B2 H12 T777, 50 for B1 H16 T32768, whose 16
// workgroups take 4096 rows a round.
constexpr int kDgThreads = 1024;

// x of another lane by a DPP move (0 where there is none), halves of a double
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_f64(double x) {
  u32x2 w = __builtin_bit_cast(u32x2, x);
  w[0] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROWS, 0xF, false);
  w[1] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, w);
}
__device__ __forceinline__ double lane_f64(double x, int lane) {
  u32x2 w = __builtin_bit_cast(u32x2, x);
  w[0] = (uint32_t)__builtin_amdgcn_readlane((int)w[0], lane);
  w[1] = (uint32_t)__builtin_amdgcn_readlane((int)w[1], lane);
  return __builtin_bit_cast(double, w);
}
// sum over the lanes up to this one
__device__ __forceinline__ double wave_prefix_f64(double x) {
  x += dpp_f64<0x111>(x);   // row_shr:1, 2, 4, 8, then the last lanes of rows into those after
  x += dpp_f64<0x112>(x);
  x += dpp_f64<0x114>(x);
  x += dpp_f64<0x118>(x);
  x += dpp_f64<0x142, 0xA>(x);
  return x + dpp_f64<0x143, 0xC>(x);
}
__device__ __forceinline__ double lane_before_f64(double x) { return dpp_f64<0x138>(x); }   // wave_shr:1

template <typename T, int CPW>
__global__ __launch_bounds__(kDgThreads) void decay_grad_kernel(const float* dotq, const float* dotk, int slices,
                                                                const T* gate, const float* dhT, const float* hT,
                                                                int elems, int has_h0, const int* lens, int rows, int heads,
                                                                T* dg, double* head_sum, int head_decay) {
  constexpr int WAVES = kDgThreads / 64, NC = WAVES * CPW;   // chunks of a round
  static_assert(NC <= 64, "one lane of the wave that runs X per chunk");
  __shared__ double s_wave[WAVES], s_x[NC];
  __shared__ float s_a[NC], s_b[NC], s_size[NC], s_whole[NC];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  // sum over the workgroup, for wave 0
  auto total = [&](double x) __attribute__((always_inline)) {
    x = wave_prefix_f64(x);
    if (lane == 63) s_wave[wave] = x;
    __syncthreads();
    x = 0.0;
    if (wave == 0)
      for (int w = 0; w < WAVES; ++w) x += s_wave[w];
    return x;
  };
  const int bh = blockIdx.x;
  const int len = lens ? min(max(lens[bh / heads], 0), rows) : rows;
  const int nch = (len + C - 1) / C;
  const T* gp = gate + (head_decay ? (size_t)(bh % heads) : (size_t)bh * rows);
  // wave 0: X of the chunk after a round's first, and that chunk's sum of a and size
  double x_after = 0.0, a_after = 0.0, sum = 0.0;
  float size_after = 0.f;
  if (dhT) {
    double y = 0.0;
    const f32x4 *p = reinterpret_cast<const f32x4*>(dhT + (size_t)bh * elems),
                *h = reinterpret_cast<const f32x4*>(hT + (size_t)bh * elems);
#pragma unroll 4
    for (int i = tid; i < elems / 4; i += kDgThreads) {
      const f32x4 u = p[i], w = h[i];
      y += ((double)u[0] * w[0] + (double)u[1] * w[1]) + ((double)u[2] * w[2] + (double)u[3] * w[3]);
    }
    x_after = total(y);
  }
  const size_t half = (size_t)slices * gridDim.x * rows;   // from the dots before (after) the chunk to those in it
  for (int end = nch; end > 0; end -= NC) {   // chunks end - 1, end - 2, ..
    float mine[CPW];
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      const int i = j * WAVES + wave, c = end - 1 - i, row = C * c + lane;
      float a = 0.f, b = 0.f, in = 0.f, x = 0.f;
      if (c >= 0 && row < len) {
        x = to_f32(head_decay ? *gp : gp[row]) * kLog2E;
#pragma unroll 4   // the loads of four slices in flight
        for (int s = 0; s < slices; ++s) {
          const size_t at = ((size_t)s * gridDim.x + bh) * rows + row;
          a += dotq[at];
          b += dotk[at];
          in += dotq[half + at] - dotk[half + at];
        }
      }
      const bool closed = x < -126.f;
      const unsigned long long shut = __ballot(closed);
      const float from = wave_suffix(a, lane), upto = wave_prefix(b), before = lane_before(upto);
      float tail = wave_suffix(in, lane);
      if (shut) {   // pairs in the chunk: of the rows up to the next closed gate
        const unsigned long long later = lane < 63 ? shut >> (lane + 1) : 0;
        // (summed again for that: a difference of tails would keep the rounding of what lies behind the gate)
        tail = in;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const float y = __shfl_down(tail, off, 64);
          if (lane + off < 64 && (later & ((1ull << off) - 1)) == 0) tail += y;
        }
      }
      mine[j] = closed ? 0.f : from + before + tail;
      const float size = group_sum<64>(fabsf(a) + fabsf(b));
      const float whole = group_sum<64>(x < kDecayFloor ? kDecayFloor : x);   // log2 of the chunk's decay
      if (lane == 0) {
        s_a[i] = from;
        s_size[i] = size;
        s_whole[i] = shut ? kDecayFloor : whole;
      }
      if (lane == 63) s_b[i] = upto;
    }
    __syncthreads();
    if (wave == 0) {
      constexpr float kNoise = sizeof(T) == 2 ? 0x1p-19f : 0x1p-23f;
      const int n = min(end, NC), c = end - 1 - lane;   // a lane a chunk
      const bool live = lane < n, last = c == nch - 1;
      const double a = live ? s_a[lane] : 0.0, b = live ? s_b[lane] : 0.0;
      const float size = live ? s_size[lane] : 0.f, whole = live ? s_whole[lane] : 0.f;
      double a_prev = lane_before_f64(a);
      float size_prev = __shfl_up(size, 1, 64);
      if (lane == 0) a_prev = a_after, size_prev = size_after;
      double x = live && !last ? a_prev - b : 0.0;
      if (lane == 0) x += x_after;
      x = wave_prefix_f64(x);
      // the first chunk that starts anew, then the first one after it, ..
      const bool zero = whole < -126.f || (c == 0 && !has_h0), faint = whole < -16.f && !last;
      const double noise = (double)(kNoise * fmaxf(size, size_prev));
      double base = 0.0;
      int done = -1;
      for (;;) {
        const unsigned long long hit = __ballot(live && lane > done && (zero || (faint && fabs(x - base) <= noise)));
        if (!hit) break;
        done = __ffsll((long long)hit) - 1;
        const double at = lane_f64(x, done);
        if (lane >= done) base = at;
      }
      x -= base;
      if (live) s_x[lane] = x;
      x_after = lane_f64(x, n - 1);
      a_after = lane_f64(a, n - 1);
      size_after = __shfl(size, n - 1, 64);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < CPW; ++j) {
      const int i = j * WAVES + wave, c = end - 1 - i, row = C * c + lane;
      if (c < 0 || row >= len) continue;
      const double d = mine[j] + s_x[i];
      if (head_decay) sum += d;
      else dg[(size_t)bh * rows + row] = from_f32<T>((float)d);
    }
    __syncthreads();   // before the next round's sums
  }
  if (head_decay) {
    __syncthreads();
    sum = total(sum);
    if (tid == 0) {
      if (head_sum) head_sum[blockIdx.x] = sum;
      else dg[blockIdx.x] = from_f32<T>((float)sum);
    }
  }
}

// The second kernel of a constant decay's gradient: one thread per head.
template <typename T>
__device__ __forceinline__ void add_batches(const double* head_sum, int B, int H, T* dg) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  if (h >= H) return;
  double x = 0.0;
#pragma unroll 8
  for (int b = 0; b < B; ++b) x += head_sum[(size_t)b * H + h];
  dg[h] = from_f32<T>((float)x);
}
template <typename T>
__global__ __launch_bounds__(256) void head_decay_grad_kernel(const double* head_sum, int B, int H, T* dg) {
  add_batches(head_sum, B, H, dg);
}

// Gradients of a query or key shared by `group` heads: the sum of the heads'
// fp32 parts [units, group, rows, d], rounded once.  Four elements per thread.
// HBM-bound: 112 us for the 600 MB of B1 H16 Hk4 T32768 d128.  A third plane of
// workgroups takes add_batches() along, which saves a launch (2 to 5 us).
template <typename T>
__global__ __launch_bounds__(256) void fold_heads_kernel(const float* qparts, const float* kparts, int units, int group,
                                                         int rows, int d, const int* lens, int units_per_batch, T* dq,
                                                         T* dk, const double* head_sum, int B, int H, T* dg) {
  if (blockIdx.y == 2) return add_batches(head_sum, B, H, dg);
  const float* parts = blockIdx.y ? kparts : qparts;
  T* out = blockIdx.y ? dk : dq;
  const long long per = (long long)rows * d;
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= units * per) return;
  const int unit = (int)(i / per);
  const long long at = i % per;
  if (lens && at / d >= lens[unit / units_per_batch]) return;
  f32x4 x = zero4();
  for (int j = 0; j < group; ++j) x += *reinterpret_cast<const f32x4*>(parts + ((long long)unit * group + j) * per + at);
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<u32x2*>(out + i) = u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
  else
    *reinterpret_cast<f32x4*>(out + i) = x;
}

// ---------------------------------------------------------------- one token
// H <- a H + k v^T, o = H^T q, one read and one write of the state.  A
// workgroup holds DVS columns of one state: each thread 16-byte columns of
// ITER rows in registers, stored as soon as they are updated; the column sums
// of q_i H_i go through LDS.  HBM-bound: 220 us for 8192 states of 128 x 128
// (4.9 TB/s, a large copy's rate; 159 us on one repeated set, which the
// last-level cache holds half of).
constexpr int kLaDecodeThreads = 256;

template <typename T, int DK, int DVS>
__global__ __launch_bounds__(kLaDecodeThreads) void linattn_decode_kernel(const T* __restrict__ q,
                                                                          const T* __restrict__ k,
                                                                          const T* __restrict__ v,
                                                                          const T* __restrict__ gate, float* __restrict__ H,
                                                                          T* __restrict__ o, int heads, int group, int dv,
                                                                          int head_decay) {
  constexpr int TPR = DVS / 4;
  constexpr int RPI = kLaDecodeThreads / TPR;
  constexpr int ITER = (DK + RPI - 1) / RPI;
  __shared__ float s_k[DK], s_q[DK];
  __shared__ f32x4 s_o[RPI][TPR];
  const int slices = dv / DVS;
  const long long st = blockIdx.x / slices;
  const int col0 = (int)(blockIdx.x % slices) * DVS;
  const int tid = threadIdx.x, cg = tid % TPR, rg = tid / TPR;
  float* Hs = H + st * (long long)DK * dv + col0 + 4 * cg;
  f32x4 h[ITER];
#pragma unroll
  for (int j = 0; j < ITER; ++j) {
    const int row = rg + j * RPI;
    if (row < DK) h[j] = *reinterpret_cast<const f32x4*>(Hs + row * dv);
  }
  const long long kh = st / group;   // the state's query and key head
  for (int i = tid; i < DK; i += kLaDecodeThreads) {
    s_k[i] = to_f32(k[kh * DK + i]);
    s_q[i] = to_f32(q[kh * DK + i]);
  }
  f32x4 vv;
#pragma unroll
  for (int e = 0; e < 4; ++e) vv[e] = to_f32(v[st * dv + col0 + 4 * cg + e]);
  // a slow decay by its distance from 1, as in decay_less_one: rounded to fp32 it
  // would move a long memory to one side, token by token
  const float x = to_f32(gate[head_decay ? st % heads : st]);
  const float a = expf(x), less = fabsf(x) < 0.35f ? expm1f(x) : 0.f;
  __syncthreads();
  f32x4 acc = zero4();
#pragma unroll
  for (int j = 0; j < ITER; ++j) {
    const int row = rg + j * RPI;
    if (row < DK) {
      f32x4 hn;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        hn[e] = (less != 0.f ? __builtin_fmaf(h[j][e], less, h[j][e]) : a * h[j][e]) + s_k[row] * vv[e];
      acc += s_q[row] * hn;
      // streaming store: the state is not read again in this step
      __builtin_nontemporal_store(hn, reinterpret_cast<f32x4*>(Hs + row * dv));
    }
  }
  s_o[rg][cg] = acc;
  __syncthreads();
  // column c of the slice: its RPI partial sums
  for (int c = tid; c < DVS; c += kLaDecodeThreads) {
    float x = 0.f;
#pragma unroll 8
    for (int i = 0; i < RPI; ++i) x += s_o[i][c / 4][c % 4];
    o[st * dv + col0 + c] = from_f32<T>(x);
  }
}

template <typename T, int DK, int DVS>
static hipError_t launch_la_decode_t(const LinAttnDecodeArgs& a) {
  const long long wgs = (long long)a.N * a.H * (a.dv / DVS);
  hipLaunchKernelGGL((linattn_decode_kernel<T, DK, DVS>), dim3((unsigned)wgs), dim3(kLaDecodeThreads), 0, a.stream,
                     (const T*)a.q, (const T*)a.k, (const T*)a.v, (const T*)a.g, a.H_inout, (T*)a.o, a.H, a.H / a.Hk,
                     a.dv, a.head_decay);
  return hipGetLastError();
}

template <typename T, int DK>
static hipError_t la_decode_dvs(const LinAttnDecodeArgs& a, int dvs) {
  switch (dvs) {
    case 16: return launch_la_decode_t<T, DK, 16>(a);
    case 32: return launch_la_decode_t<T, DK, 32>(a);
    case 64: return launch_la_decode_t<T, DK, 64>(a);
    case 128: return launch_la_decode_t<T, DK, 128>(a);
  }
  return hipErrorInvalidValue;
}

template <typename T>
static hipError_t la_decode_dk(const LinAttnDecodeArgs& a, int dvs) {
  switch (a.dk) {
    case 16: return la_decode_dvs<T, 16>(a, dvs);
    case 32: return la_decode_dvs<T, 32>(a, dvs);
    case 64: return la_decode_dvs<T, 64>(a, dvs);
    case 128: return la_decode_dvs<T, 128>(a, dvs);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_linattn_decode(const LinAttnDecodeArgs& a) {
  const long long states = (long long)a.N * a.H;
  if (states == 0) return hipSuccess;
  // Few states: their columns over more CUs, down to 32 (rows of 128 bytes).
  // us on one repeated set of states, bf16 d128, whole | to 32 | to 16 columns:
  // 16 states 3.7 | 3.2 | 3.8, 32 states 3.8 | 3.3 | 4.4, 64 states 4.1 | 3.6, 128 states 4.6 | 4.2
  int dvs = a.dv;
  while (dvs > 32 && states * (a.dv / dvs) < 256) dvs /= 2;
  return a.dtype == 1 ? la_decode_dk<bf16_t>(a, dvs) : la_decode_dk<float>(a, dvs);
}

// ---------------------------------------------------------------- host side

static hipError_t launch_sweep(const SweepLaunch& L, int dtype, int d1, int ds, hipStream_t stream) {
  return dtype == 1 ? launch_sweep_e<bf16_t>(L, d1, ds, stream) : launch_sweep_e<float>(L, d1, ds, stream);
}

// How a call is split over workgroups: slices of `ds` value columns (of the
// widths that has more), and segments of rows, whose start states come from
// the segments' own states (own_state_kernel reads y and z once more) joined in
// order; the own states are formed over sub-segments, short enough to occupy
// the CUs as well.
//
// Wide slices do the work that does not depend on the columns (Y X^T, its
// decays, the copies of Y) fewer times, narrow ones and segments give a call
// of few heads more workgroups.  The split is the one of least time by the
// measured time of a chunk (MI355X, 256 workgroups, us; d2 = 128):
//   bf16, d1 128:  1.39, 1.77, 2.82, 4.97 for slices of 16, 32, 64, 128 columns
//         d1 64:   1.17, 1.46, 1.92, 3.69      d1 32:  1.00, 1.26, 1.64, 3.53
//   fp32, d1 128:  4.10, 5.43, 8.50 (16, 32, 64; wider ones do not fit in LDS)
//         d1 64:   2.52, 3.24, 4.87            d1 32:  1.73, 2.34, 3.45
// to which chunk_us() is fitted.
//
// A backward of different widths has two launches, one contracting over dk and
// two sweeps over dv; with few heads one launch of all three, the narrower
// contraction padded with zeros, fills the CUs better (us, two launches -> one:
// bf16 B2 H12 T777 dk64 dv128 40.0 -> 31.8, B1 H8 T2000 dk32 dv64 34.7 -> 31.4,
// fp32 B3 H8 T1000 dk64 dv128 94.7 -> 83.8).  With slices wider than
// kPadSlice the launches are full anyway.
struct Split {
  int ds;
  int seg_rows, nseg, sub_rows, subs, nsub;   // subs: sub-segments per segment; nsub: of the whole sequence
  bool together;   // backward of different widths: the sweeps in one launch, the narrower contraction padded
};
static double chunk_us(int d1, int ds, int dtype) {
  return dtype == CKDA_DTYPE_BF16 ? 0.8 + ds * (0.009 + 0.00018 * d1) : 0.7 + 0.015 * d1 + ds * (0.017 + 0.00059 * d1);
}
// a segment's first loads and its start state
static double segment_us(int d1, int ds) { return 2.5 + 0.00015 * d1 * ds; }
static double own_chunk_us(int d1, int d2, int dtype) {
  return dtype == CKDA_DTYPE_BF16 ? 0.5 + 0.00006 * d1 * d2 : 0.6 + 0.0003 * d1 * d2;
}
static int slice_width(int d2, int ds) { return std::min(d2, ds); }

// dk, dv: widths; backward: the three gradient sweeps (and both directions'
// segment states) instead of the forward one
static Split plan_split(long long heads, int T, int dk, int dv, int dtype, bool backward) {
  constexpr long long kCUs = 256;
  const int nch = std::max(1, (T + C - 1) / C);
  const long long dirs = backward ? 2 : 1;
  Split best = {};
  double least = 0.0;
  for (int ds = 16; ds <= (dtype == CKDA_DTYPE_BF16 ? 128 : 64); ds *= 2) {
    if (ds > 16 && ds > std::max(dk, dv)) break;
    const long long sk = dk / slice_width(dk, ds), sv = dv / slice_width(dv, ds);
    const long long wgs = heads * (backward ? 2 * sk + sv : sv);
    // segments: none, two, three, or as many as fill the CUs once to four times
    // (short sequences and full grids: none)
    for (int i = 0; i < (nch < 4 || wgs >= 2 * kCUs ? 1 : 7); ++i) {
      const long long n = i < 3 ? i + 1 : kCUs * (i - 2) / std::max(1LL, wgs);
      if (n < 1) continue;
      Split p;
      p.ds = ds;
      int per = (int)((nch + n - 1) / n);   // chunks of a segment
      if (n > 1 && per < 2) break;
      p.nseg = (nch + per - 1) / per;
      // sub-segments: two workgroups per CU, at least two chunks each
      long long subs = 1;
      if (p.nseg > 1 && heads > 0)
        subs = std::max(1LL, std::min(2 * kCUs / std::max(1LL, dirs * heads * (p.nseg - 1)), (long long)per / 2));
      const int sub = (int)((per + subs - 1) / subs);
      p.subs = (per + sub - 1) / sub;
      per = p.subs * sub;   // whole sub-segments
      p.nseg = (nch + per - 1) / per;
      p.together = false;
      p.sub_rows = sub * C;
      p.seg_rows = per * C;
      p.nsub = (p.nseg - 1) * p.subs + 1;   // the last segment's start is the last one needed
      auto rounds = [&](long long wgs, long long at_once) { return (double)((wgs + at_once - 1) / at_once); };
      auto sweep = [&](long long slices, int d1, int d2) {
        return rounds(heads * slices * p.nseg, kCUs) *
               (segment_us(d1, slice_width(d2, ds)) + per * chunk_us(d1, slice_width(d2, ds), dtype));
      };
      double us = !backward ? sweep(sv, dk, dv) : dk == dv ? sweep(2 * sk + sv, dk, dv) : sweep(sv, dk, dv) + sweep(2 * sk, dv, dk) + 2.0;
      if (backward && dk != dv && ds <= kPadSlice && std::min(dk, dv) >= ds) {
        const double one = sweep(2 * sk + sv, std::max(dk, dv), ds);   // (a slice's width counts, not d2)
        if ((p.together = one < us)) us = one;
      }
      if (p.nseg > 1) {
        // two launches more: the own states (two workgroups a CU take some 1.6
        // times as long as one), and one pass over the states.
        const double own = rounds(dirs * heads * (p.nsub - 1), 2 * kCUs) * sub * own_chunk_us(dk, dv, dtype) * 1.6;
        us += 8.0 + own + (double)dirs * heads * p.nsub * dk * dv * 8 / 4e6;
        // Segments have to promise a tenth less: chunks of a launch that leaves
        // CUs idle take less than the times above, which the model does not know.
        // One call stands behind the tenth: the backward of B4 H16 T4096 d128, bf16
        // (192 workgroups of whole sequences 235 us in all when this was measured,
        // four segments, estimated at 98% of that, 285 us)
        us *= 1.1;
      }
      if (best.ds == 0 || us < least) {
        best = p;
        least = us;
      }
    }
  }
  return best;
}

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// workspace of the forward: the sub-segments' states and decays
struct FwdPlan {
  Split sp;
  size_t states, decay, bytes;
};
static FwdPlan fwd_plan(int B, int H, int T, int dk, int dv, int dtype) {
  FwdPlan p;
  const size_t bh = (size_t)B * H;
  p.sp = plan_split((long long)bh, T, dk, dv, dtype, false);
  p.states = 0;
  p.decay = p.sp.nseg > 1 ? up256((size_t)p.sp.nsub * bh * dk * dv * 4) : 0;
  p.bytes = p.sp.nseg > 1 ? p.decay + up256((size_t)p.sp.nsub * bh * 8) : 0;
  return p;
}
size_t linattn_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, int dtype) {
  return fwd_plan(B, H, T, dk, dv, dtype).bytes;
}

static SweepLaunch sweep_base(const LinAttnArgs& a) {
  SweepLaunch L = {};
  L.units = a.B * a.Hk;
  L.group = a.H / a.Hk;
  L.heads = a.H;
  L.rows = a.T;
  L.lens = a.lens;
  L.g = a.g;
  L.head_decay = a.head_decay;
  return L;
}

static void set_split(SweepLaunch& L, const LinAttnArgs& a, const Split& sp) {
  L.seg_rows = sp.seg_rows;
  L.nseg = sp.nseg;
  L.seg_subs = sp.subs;
  L.seg_stride = (long long)a.B * a.H * a.dk * a.dv;
}

// the states at the starts of all sub-segments: forward in time and, with
// rstates, backward in time, both in the same launches (the whole backward, two
// pairs of launches -> one: fp32 B1 H8 T1023 d64 38.6 -> 31.1 us, bf16 B1 H8
// T4096 d128 98 -> 72, B1 H4 T8192 d64 63 -> 46)
static hipError_t segment_starts(const LinAttnArgs& a, const Split& sp, float* states, float2* decay, float* rstates,
                                 float2* rdecay) {
  SweepLaunch L = sweep_base(a);
  set_split(L, a, sp);
  L.seg_rows = sp.sub_rows;
  L.nroles = rstates ? 2 : 1;
  SweepRole &F = L.role[0], &R = L.role[1];
  F.y = a.k;
  F.z = a.v;
  F.seg_out = states;
  F.seg_decay = decay;
  F.drop_end = rstates != nullptr;   // (the backward's dq sweep)
  R.y = a.q;
  R.z = a.dout;
  R.seg_out = rstates;
  R.seg_decay = rdecay;
  R.reverse = 1;
  F.y_shared = R.y_shared = 1;
  F.d2 = R.d2 = a.dv;
  L.nseg = sp.nsub - 1;   // (the last one's own state is not needed)
  L.parts = L.nroles * L.group;
  hipError_t e = a.dtype == 1 ? launch_own_e<bf16_t>(L, a.dk, a.stream) : launch_own_e<float>(L, a.dk, a.stream);
  if (e != hipSuccess) return e;
  const long long threads = L.seg_stride / 4;
  hipLaunchKernelGGL(segment_scan_kernel, dim3((unsigned)((threads + 255) / 256), L.nroles), dim3(256), 0, a.stream,
                     ScanArgs{states, decay, a.h0}, ScanArgs{rstates, rdecay, a.dhT}, sp.nsub, a.B * a.H,
                     (long long)a.dk * a.dv, L.seg_stride);
  return hipGetLastError();
}

hipError_t launch_linattn_fwd(const LinAttnArgs& a) {
  const FwdPlan p = fwd_plan(a.B, a.H, a.T, a.dk, a.dv, a.dtype);
  unsigned char* ws = (unsigned char*)a.workspace;
  float* states = (float*)(ws + p.states);
  if (p.sp.nseg > 1) {
    hipError_t e = segment_starts(a, p.sp, states, (float2*)(ws + p.decay), nullptr, nullptr);
    if (e != hipSuccess) return e;
  }
  SweepLaunch L = sweep_base(a);
  const int ds = slice_width(a.dv, p.sp.ds);
  set_split(L, a, p.sp);
  L.nroles = 1;
  SweepRole& R = L.role[0];
  R.x = a.q;
  R.y = a.k;
  R.x_shared = R.y_shared = 1;
  R.z = a.v;
  R.d1 = a.dk;
  R.d2 = a.dv;
  R.out = a.o;
  R.init = a.h0;
  R.fin = a.hT;
  R.seg_states = states;
  L.exact_state = a.hT != nullptr;
  R.parts = L.parts = L.group * (a.dv / ds);
  return launch_sweep(L, a.dtype, a.dk, ds, a.stream);
}

// workspace of the backward: dots of queries and keys with their gradients,
// (of either, with the rows outside and inside their chunk), the last chunk's
// decayed start state, segment states of both directions, and the heads' parts
// of shared gradients
struct BwdPlan {
  Split sp;
  size_t dotq, dotk, hT, head_sum, states, rstates, decay, dq, dk, bytes;
};
static BwdPlan bwd_plan(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  BwdPlan p;
  const size_t bh = (size_t)B * H, elems = (size_t)dk * dv;
  p.sp = plan_split((long long)bh, T, dk, dv, dtype, true);
  const int sk = dk / slice_width(dk, p.sp.ds);
  const size_t nsub = p.sp.nseg > 1 ? (size_t)p.sp.nsub : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  p.dotq = take((size_t)sk * bh * T * 8);
  p.dotk = take((size_t)sk * bh * T * 8);
  p.hT = take(bh * elems * 4);
  p.head_sum = take(bh * 8);
  p.states = take(nsub * bh * elems * 4);
  p.rstates = take(nsub * bh * elems * 4);
  p.decay = take(2 * nsub * bh * 8);   // of both directions
  const bool grouped = H != Hk;
  p.dq = take(grouped ? bh * T * dk * 4 : 0);
  p.dk = take(grouped ? bh * T * dk * 4 : 0);
  p.bytes = at;
  return p;
}
size_t linattn_bwd_workspace_bytes(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  return bwd_plan(B, H, Hk, T, dk, dv, dtype).bytes;
}

// A launch takes fewer than 2^32 threads.
bool linattn_fits_grid(int B, int H, int Hk, int T, int dk, int dv, int dtype, bool backward) {
  const long long bh = (long long)B * H, units = (long long)B * Hk;
  long long most = 0;
  if (bh > 65536) {   // (fewer heads have at most 24 slices each, or some 2000 segments among them)
    const Split sp = plan_split(bh, T, dk, dv, dtype, backward);
    const long long sk = dk / slice_width(dk, sp.ds), sv = dv / slice_width(dv, sp.ds);
    const long long slices = backward ? sv + 2 * sk : sv;
    most = std::max(512 * cell_workgroups(units * sp.nseg, (int)(H / Hk * slices)), backward ? kDgThreads * bh : 0);
  }
  if (backward && H != Hk) most = std::max(most, units * T * (dk / 4));   // fold_heads_kernel
  return most + 255 <= (long long)UINT32_MAX;
}

template <typename T>
static hipError_t launch_bwd_tail(const LinAttnArgs& a, const BwdPlan& p, unsigned char* ws) {
  const int bh = a.B * a.H, slices = a.dk / slice_width(a.dk, p.sp.ds);
  double* sums = a.head_decay && a.B != 1 ? (double*)(ws + p.head_sum) : nullptr;
  hipError_t e = hipSuccess;
  if (bh > 0) {
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(bh), dim3(kDgThreads), 0, a.stream, (const float*)(ws + p.dotq),
                         (const float*)(ws + p.dotk), slices, (const T*)a.g, a.dhT, (const float*)(ws + p.hT), a.dk * a.dv,
                         a.h0 != nullptr, a.lens, a.T, a.H, (T*)a.dg, sums, a.head_decay);
    };
    a.T <= kDgThreads ? launch(decay_grad_kernel<T, 1>) : launch(decay_grad_kernel<T, 4>);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const unsigned head_blocks = (a.H + 255) / 256;
  if (a.H != a.Hk && bh > 0 && a.T > 0) {
    const int units = a.B * a.Hk;
    const long long threads = (long long)units * a.T * a.dk / 4;
    const unsigned blocks = std::max((unsigned)((threads + 255) / 256), sums ? head_blocks : 0u);
    hipLaunchKernelGGL((fold_heads_kernel<T>), dim3(blocks, sums ? 3 : 2), dim3(256), 0, a.stream,
                       (const float*)(ws + p.dq), (const float*)(ws + p.dk), units, a.H / a.Hk, a.T, a.dk, a.lens, a.Hk,
                       (T*)a.dq, (T*)a.dk_out, sums, a.B, a.H, (T*)a.dg);
    e = hipGetLastError();
  } else if (sums) {
    hipLaunchKernelGGL((head_decay_grad_kernel<T>), dim3(head_blocks), dim3(256), 0, a.stream, sums, a.B, a.H, (T*)a.dg);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_linattn_bwd(const LinAttnArgs& a) {
  const BwdPlan p = bwd_plan(a.B, a.H, a.Hk, a.T, a.dk, a.dv, a.dtype);
  unsigned char* ws = (unsigned char*)a.workspace;
  float *states = (float*)(ws + p.states), *rstates = (float*)(ws + p.rstates);
  hipError_t e;
  if (p.sp.nseg > 1) {
    float2 *decay = (float2*)(ws + p.decay), *rdecay = decay + (size_t)p.sp.nsub * a.B * a.H;
    if ((e = segment_starts(a, p.sp, states, decay, rstates, rdecay)) != hipSuccess) return e;
  }
  const bool grouped = a.H != a.Hk;
  const int dsk = slice_width(a.dk, p.sp.ds), dsv = slice_width(a.dv, p.sp.ds);
  SweepRole dv = {}, dk = {}, dq = {};
  dv.x = a.k;
  dv.y = a.q;
  dv.x_shared = dv.y_shared = 1;
  dv.z = a.dout;
  dv.d1 = a.dk;
  dv.d2 = a.dv;
  dv.reverse = 1;
  dv.out = a.dv_out;
  dv.init = a.dhT;
  dv.fin = a.dh0;
  dv.seg_states = rstates;
  dk.x = a.v;
  dk.y = a.dout;
  dk.z = dq.w = a.q;
  dk.w = dq.z = a.k;
  dk.z_shared = dk.w_shared = dq.z_shared = dq.w_shared = 1;
  dk.d1 = dq.d1 = a.dv;
  dk.d2 = dq.d2 = a.dk;
  dk.turned = dq.turned = 1;
  dk.reverse = 1;
  dk.out_f32 = dq.out_f32 = grouped;
  dk.out = grouped ? (void*)(ws + p.dk) : a.dk_out;
  dk.dot = (float*)(ws + p.dotk);
  dk.init = a.dhT;
  dk.seg_states = rstates;
  dq.x = a.dout;
  dq.y = a.v;
  dq.out = grouped ? (void*)(ws + p.dq) : a.dq;
  dq.dot = (float*)(ws + p.dotq);
  dq.init = a.h0;
  dq.fin = a.dhT ? (float*)(ws + p.hT) : nullptr;   // what of the last chunk's start state meets dhT
  dq.drop_end = 1;
  dq.seg_states = states;
  SweepLaunch L = sweep_base(a);
  set_split(L, a, p.sp);
  L.exact_state = a.dh0 || a.dhT;
  dv.parts = L.group * (a.dv / dsv);
  dk.parts = dq.parts = L.group * (a.dk / dsk);
  // one launch where the sweeps have the same widths or the split says so, else
  // the two that contract over dv apart from the one over dk
  if (a.dk == a.dv || p.sp.together) {
    L.role[0] = dv;
    L.role[1] = dk;
    L.role[2] = dq;
    L.nroles = 3;
    L.parts = dv.parts + dk.parts + dq.parts;
    if ((e = launch_sweep(L, a.dtype, std::max(a.dk, a.dv), dsk, a.stream)) != hipSuccess) return e;
  } else {
    L.role[0] = dv;
    L.nroles = 1;
    L.parts = dv.parts;
    if ((e = launch_sweep(L, a.dtype, a.dk, dsv, a.stream)) != hipSuccess) return e;
    L.role[0] = dk;
    L.role[1] = dq;
    L.nroles = 2;
    L.parts = dk.parts + dq.parts;
    if ((e = launch_sweep(L, a.dtype, a.dv, dsk, a.stream)) != hipSuccess) return e;
  }
  return a.dtype == 1 ? launch_bwd_tail<bf16_t>(a, p, ws) : launch_bwd_tail<float>(a, p, ws);
}

}  // namespace ckda
