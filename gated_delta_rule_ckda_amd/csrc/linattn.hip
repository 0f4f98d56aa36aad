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
// state slice in their accumulators and copy the next chunk's operands into
// LDS.  Everything is double buffered, one barrier a chunk:
//   output waves:  S^T = Y X^T tile by tile (rows s, columns t), P^T = G . S^T
//                  in fp32 on the accumulators, which are then, in the K order
//                  of ckda_device.hpp, the B operand of Z^T P^T; exp(c_t)
//                  scales the accumulators of H^T X^T (a factor of the column);
//   state waves:   H <- exp(c_C) H + Y^T (G(C, .) Z), then the new H^T to LDS;
//   copy waves:    Y, Z and the terms of G(C, .) Z of the next chunk, the decay
//                  factors of the one after it.
// Precision: the inputs are exact in bf16; every factor that is not (P, H and
// the scaled Z) is carried as a sum of bf16 terms: two (16 bits) where the
// product ends in a rounded output, three (24 bits) for the state itself,
// which is returned in fp32.  All sums are fp32.  fp32 inputs take the fp32
// matrix cores throughout.
// Log decays are summed as two parts, whole multiples of 1/64 (whose sums are
// exact) and the rest, so that differences of large sums keep fp32 accuracy.
#include <type_traits>

#include "ckda_device.hpp"
#include "ckda_internal.hpp"

namespace ckda {

namespace {

constexpr int C = kLaChunk;    // rows of a chunk
constexpr int RT = C / 16;     // row tiles

template <typename T, int D1, int DS, bool OUT, bool EXACT>
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
  // four state waves: wave w owns column tile w % NDV, row tiles (w / NDV) TPW ..
  static constexpr int WPC = 4 / NDV;                // waves on one column tile
  static constexpr int TPW = (RH + WPC - 1) / WPC;   // row tiles per wave
  static constexpr int Y_BYTES = C * YROW, Z_BYTES = C * ZROW, H_BYTES = DS * YROW;
  static constexpr int HSETS = BF ? 2 : 1;           // terms of H: hi and lo
  static constexpr int ZSETS = BF ? (EXACT ? 3 : 2) : 1;   // terms of the scaled Z
  // one of two operand sets: Y, Z, the terms of G(C, .) Z, the terms of H^T
  static constexpr int Z_OFF = Y_BYTES, ZS_OFF = Z_OFF + Z_BYTES, H_OFF = ZS_OFF + ZSETS * Z_BYTES;
  static constexpr int SET = H_OFF + (OUT ? HSETS * H_BYTES : 0);
  // one of four sets of decay factors: c (whole), c (rest), exp(c_t), G(C, t), G(tile end, t)
  static constexpr int DEC_BYTES = 5 * C * 4, DEC_OFF = 2 * SET;
  static constexpr int LDS_BYTES = DEC_OFF + 4 * DEC_BYTES;
  // pieces of 16 bytes that the 256 threads of the state waves copy
  static constexpr int YPR = D1 * E / 16, ZPR = ZROW / 16;
  static constexpr int NY = (C * YPR + 255) / 256, NZ = (C * ZPR + 255) / 256;
};

// Byte offset of the 16-byte piece `piece` of row `row` in an LDS array of
// ROWB-byte rows.  The piece index is xor-ed with twice the number of the
// row's 256-byte line, so that neither kind of operand read has bank conflicts
// (SQ_LDS_BANK_CONFLICT 0): a transposing 8-byte read takes 32 bytes of 8 rows
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

// rows row0 + r, K block kb along the row
template <int ROWB>
__device__ __forceinline__ Frag row_frag(const unsigned char* m, int row0, int kb, int g, int r) {
  return load_frag(m + lds_piece<ROWB>(row0 + r, kb * 4 + g));
}

// column col0 + r, rows of K block kb in the K order kappa
template <typename T, int ROWB>
__device__ __forceinline__ Frag col_frag(const unsigned char* m, int col0, int kb, int g, int r) {
  Frag f;
  if constexpr (sizeof(T) == 2) {
    // two transposing reads (ds_read_b64_tr_b16): within 16 lanes, lane i gets
    // as element j the element i % 4 of the 8 bytes lane 4 j + i / 4 addresses
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const int row = kb * 32 + 4 * g + (r >> 2), piece = col0 / 8 + ((r & 3) >> 1), half = (r & 1) * 8;
    const u32x2 a = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(m + lds_piece<ROWB>(row, piece) + half)));
    const u32x2 b = __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(m + lds_piece<ROWB>(row + 16, piece) + half)));
    f.w = u32x4{a[0], a[1], b[0], b[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f.w[e] = *reinterpret_cast<const uint32_t*>(m + lds_piece<ROWB>(kb * 16 + 4 * g + e, (col0 + r) / 4) +
                                                  ((col0 + r) % 4) * 4);
  }
  return f;
}

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

// the value of lane 15 of this lane's row of 16 (DPP row_newbcast)
__device__ __forceinline__ float row_last(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x15F, 0xF, 0xF, false));
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kDecayFloor = -240.f;   // 2^-240 is 0 in fp32, and 64 such steps keep their sum's parts exact

// three bf16 terms of x: hi + mid + lo = x to 2^-25 of |x|
__device__ __forceinline__ void split3_bf16(const float* v, Frag& fh, Frag& fm, Frag& fl) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = v[2 * i], b = v[2 * i + 1];
    uint32_t h = pack_bf16x2(a, b);
    asm("" : "+v"(h));
    const float ra = a - bf16_lo_half(h), rb = b - bf16_hi_half(h);
    uint32_t m = pack_bf16x2(ra, rb);
    asm("" : "+v"(m));
    fh.w[i] = h;
    fm.w[i] = m;
    fl.w[i] = pack_bf16x2(ra - bf16_lo_half(m), rb - bf16_hi_half(m));
  }
}

// OUT: with output waves (768 threads); without, only the states (512).
// EXACT: states with three bf16 terms (one is returned), else two.
template <typename T, int D1, int DS, bool OUT, bool EXACT>
__global__ __launch_bounds__(OUT ? 768 : 512) void sweep_kernel(SweepLaunch L) {
  using S = SweepCfg<T, D1, DS, OUT, EXACT>;
  constexpr int E = S::E, KBN = S::KBN, KBC = S::KBC, NDV = S::NDV, TPW = S::TPW;
  constexpr bool BF = S::BF;
  __shared__ __attribute__((aligned(16))) unsigned char lds[S::LDS_BYTES];

  const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
  const int g = lane / 16, r = lane % 16;

  // workgroup -> unit (key head of a batch entry) and its part of it: role,
  // segment, head of the group, slice.  A unit's parts get ids equal modulo 8
  // where the units allow it, so that they share an XCD's L2.
  int unit, part;
  {
    const int id = blockIdx.x;
    if (L.units % 8 == 0) {
      unit = (id / 8) / L.parts * 8 + id % 8;
      part = (id / 8) % L.parts;
    } else {
      unit = id / L.parts;
      part = id % L.parts;
    }
  }
  int role = 0;
  while (role + 1 < L.nroles && part >= L.role[role].parts) part -= L.role[role++].parts;
  const SweepRole A = L.role[role];
  const int slices = A.d2 / DS;
  const int slice = part % slices;
  const int bh = unit * L.group + (part / slices) % L.group;
  const int seg = part / slices / L.group;

  const int len = L.lens ? min(max(L.lens[bh / L.heads], 0), L.rows) : L.rows;
  const int row0 = seg * L.seg_rows;
  const int nrows = min(max(len - row0, 0), L.seg_rows);
  const int nch = (nrows + C - 1) / C, last = max(nch - 1, 0);
  // LDS row j of chunk c is row row0 + 64 c + j of the sweep: that row of the
  // sequence, or the len - 1 - that one.  Rows outside [0, len) fall outside
  // the buffers below: they read as zero and are not stored.
  const int dir = A.reverse ? -1 : 1;
  const int first = A.reverse ? len - 1 - row0 : row0;
  auto head = [&](int shared) __attribute__((always_inline)) { return (size_t)(shared ? unit : bh); };
  auto rows_rsrc = [&](const void* p, int shared, int width, int es) __attribute__((always_inline)) {
    return make_rsrc((const unsigned char*)p + head(shared) * L.rows * width * es, (uint32_t)(len * width * es));
  };
  // this head's log decays
  const T* gp = (const T*)L.g + (L.head_decay ? (size_t)(bh % L.heads) : (size_t)bh * L.rows);
  auto set_of = [&](int c) __attribute__((always_inline)) { return lds + (c & 1) * S::SET; };
  auto dec_of = [&](int c) __attribute__((always_inline)) {
    return reinterpret_cast<float*>(lds + S::DEC_OFF + (c & 3) * S::DEC_BYTES);
  };
  constexpr int Z_OFF = S::Z_OFF, ZS_OFF = S::ZS_OFF, H_OFF = S::H_OFF;

  if (OUT && wave < 4) {
    // ============================================================ output waves
    const __amdgpu_buffer_rsrc_t xr = rows_rsrc(A.x, A.x_shared, D1, E);
    const int oes = A.out_f32 ? 4 : E;
    const __amdgpu_buffer_rsrc_t outr = rows_rsrc(A.out, 0, A.d2, oes);
    const __amdgpu_buffer_rsrc_t wr = rows_rsrc(A.w, A.w_shared, A.d2, A.w ? E : 0);
    const int t = 16 * wave + r;      // this lane's row of the chunk
    Frag x0[KBN], x1[KBN];            // this chunk's rows and the next one's
    u32x4 w0[NDV], w1[NDV];           // four elements each
    auto load_x = [&](int c, Frag* d, u32x4* w) __attribute__((always_inline)) {
      const int row = first + dir * (C * c + t);
#pragma unroll
      for (int kb = 0; kb < KBN; ++kb) {
        const int off = row * D1 * E + kb * 64 + g * 16;
        d[kb].w = __builtin_amdgcn_raw_buffer_load_b128(xr, D1 < S::KB && g * 16 >= D1 * E ? 0x7FFFFFF0 : off, 0, 0);
      }
      if (A.w) {
#pragma unroll
        for (int d2 = 0; d2 < NDV; ++d2) {
          const int off = (row * A.d2 + slice * DS + 16 * d2 + 4 * g) * E;
          if constexpr (BF) {
            const u32x2 a = __builtin_amdgcn_raw_buffer_load_b64(wr, off, 0, 0);
            w[d2] = u32x4{a[0], a[1], 0, 0};
          } else {
            w[d2] = __builtin_amdgcn_raw_buffer_load_b128(wr, off, 0, 0);
          }
        }
      }
    };
    load_x(0, x0, w0);
    lds_barrier();   // the first decay factors are there
    lds_barrier();   // set 0 is filled
    // One copy of the loop per wave: W, the wave's row tile, fixes how many
    // tiles of P it has, so the body is straight-line code.
    auto run = [&](auto wconst) __attribute__((always_inline)) {
      constexpr int W = decltype(wconst)::value;
      constexpr int NPB = (16 * W) / S::KB + 1;      // K blocks of P^T it multiplies
      constexpr int NF = S::HSETS * NDV + W + 1;     // operand fragments per K block of D1
      auto chunk = [&](int c, Frag* xf, u32x4* wv, Frag* xn, u32x4* wn) __attribute__((always_inline)) {
        const unsigned char* set = set_of(c);
        const float* dec = dec_of(c);
        load_x(min(c + 1, last), xn, wn);
        // H^T X^T and the tiles of Y X^T up to this wave's own, one K block's
        // fragments read ahead of the products
        constexpr int AHEAD = BF ? 1 : 0;   // (fp32 fragments are twice as many: none, for the registers)
        Frag f[AHEAD + 1][NF];
        auto read = [&](int kb) __attribute__((always_inline)) {
          Frag* d = f[kb & AHEAD];
#pragma unroll
          for (int i = 0; i < S::HSETS * NDV; ++i)
            d[i] = load_frag(set + H_OFF + (i / NDV) * S::H_BYTES + state_piece<S::YROW>(16 * (i % NDV) + r, kb * 4 + g));
#pragma unroll
          for (int i = 0; i <= W; ++i) d[S::HSETS * NDV + i] = row_frag<S::YROW>(set, 16 * i, kb, g, r);
        };
        f32x4 oacc[NDV], olo[NDV], p[RT];
#pragma unroll
        for (int d = 0; d < NDV; ++d) oacc[d] = olo[d] = zero4();
#pragma unroll
        for (int i = 0; i < RT; ++i) p[i] = zero4();
        if constexpr (AHEAD) read(0);
#pragma unroll
        for (int kb = 0; kb < KBN; ++kb) {
          if (kb + AHEAD < KBN) read(kb + AHEAD);
          __builtin_amdgcn_sched_barrier(0);
          const Frag* d = f[kb & AHEAD];
#pragma unroll
          for (int i = 0; i < NDV; ++i) oacc[i] = mma<T>(oacc[i], d[i], xf[kb]);
          if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < NDV; ++i) olo[i] = mma<T>(olo[i], d[NDV + i], xf[kb]);
          }
#pragma unroll
          for (int i = 0; i <= W; ++i) p[i] = mma<T>(p[i], d[S::HSETS * NDV + i], xf[kb]);
          __builtin_amdgcn_sched_barrier(0);
        }
        Frag zf[AHEAD ? NPB : 1][NDV];
#pragma unroll
        for (int kb = 0; kb < (AHEAD ? NPB : 0); ++kb)
#pragma unroll
          for (int d = 0; d < NDV; ++d) zf[kb][d] = col_frag<T, S::ZROW>(set + Z_OFF, 16 * d, kb, g, r);
        // P^T = G . (Y X^T).  Below the diagonal G(t, s) is G(t, e) G(e, s)
        // with e the last row of the tile of s: both at most 1 for decays, one
        // exponential a tile here and one a row of the chunk (state waves).
        const float ch = dec[t], cl = dec[C + t];
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float row = __builtin_amdgcn_exp2f((ch - dec[16 * i + 15]) + (cl - dec[C + 16 * i + 15]));
          const f32x4 tail = *reinterpret_cast<const f32x4*>(dec + 4 * C + 16 * i + 4 * g);
          p[i] *= tail * row;
        }
        {
          const f32x4 sh = *reinterpret_cast<const f32x4*>(dec + 16 * W + 4 * g);
          const f32x4 sl = *reinterpret_cast<const f32x4*>(dec + C + 16 * W + 4 * g);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = p[W][j] * __builtin_amdgcn_exp2f((ch - sh[j]) + (cl - sl[j]));
            p[W][j] = 4 * g + j <= r ? x : 0.f;
          }
        }
        const float gam = dec[2 * C + t];
#pragma unroll
        for (int d = 0; d < NDV; ++d) oacc[d] = (oacc[d] + olo[d]) * gam;
        // O^T += Z^T P^T
#pragma unroll
        for (int kb = 0; kb < NPB; ++kb) {
          Frag ph, pl;
          if constexpr (BF) frags_from_acc_bf16_split(p[2 * kb], p[2 * kb + 1], ph, pl);
          else ph = frag_from_acc_f32(p[kb]);
#pragma unroll
          for (int d = 0; d < NDV; ++d) {
            if constexpr (!AHEAD) zf[0][d] = col_frag<T, S::ZROW>(set + Z_OFF, 16 * d, kb, g, r);
            const Frag z = zf[AHEAD ? kb : 0][d];
            if constexpr (BF) oacc[d] = mma<T>(oacc[d], z, pl);
            oacc[d] = mma<T>(oacc[d], z, ph);
          }
        }
        // this lane holds four consecutive columns of row t
        const int row = first + dir * (C * c + t);
#pragma unroll
        for (int d = 0; d < NDV; ++d) {
          const int col = slice * DS + 16 * d + 4 * g;
          if (A.out_f32) store4<float>(outr, (row * A.d2 + col) * 4, oacc[d]);
          else store4<T>(outr, (row * A.d2 + col) * E, oacc[d]);
        }
        if (A.dot) {   // this slice's part of w_t . out_t
          float x = 0.f;
#pragma unroll
          for (int d = 0; d < NDV; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float w;
              if constexpr (BF) w = (j & 1) ? bf16_hi_half(wv[d][j >> 1]) : bf16_lo_half(wv[d][j >> 1]);
              else w = __uint_as_float(wv[d][j]);
              x = __builtin_fmaf(w, oacc[d][j], x);
            }
          x += __shfl_xor(x, 16, 64);
          x += __shfl_xor(x, 32, 64);
          if (g == 0 && (unsigned)row < (unsigned)len)
            A.dot[((size_t)slice * L.units * L.group + bh) * L.rows + row] = x;
        }
        lds_barrier();
      };
      for (int c = 0; c < nch; c += 2) {
        chunk(c, x0, w0, x1, w1);
        if (c + 1 >= nch) break;
        chunk(c + 1, x1, w1, x0, w0);
      }
    };
    switch (wave) {
      case 0: run(std::integral_constant<int, 0>{}); break;
      case 1: run(std::integral_constant<int, 1>{}); break;
      case 2: run(std::integral_constant<int, 2>{}); break;
      default: run(std::integral_constant<int, 3>{}); break;
    }
  } else if (wave < (OUT ? 8 : 4)) {
    // ============================================================ state waves
    const int sw = wave - (OUT ? 4 : 0);
    const int dvt = sw % NDV, rt0 = (sw / NDV) * TPW;   // column tile, first row tile
    // the state slice: lane (g, r) holds rows 4 g .. 4 g + 3 of column r of each of its tiles
    f32x4 h[TPW];
    const size_t sbase = (size_t)bh * D1 * A.d2;
    auto state_at = [&](int i, int j) __attribute__((always_inline)) {   // element offset inside one head's state
      const int row = 16 * (rt0 + i) + 4 * g + j, col = slice * DS + 16 * dvt + r;
      return A.turned ? col * D1 + row : row * A.d2 + col;
    };
    auto own = [&](int i) __attribute__((always_inline)) { return TPW * S::WPC == S::RH || rt0 + i < S::RH; };
    const float* init = L.nseg > 1 ? (A.seg_states ? A.seg_states + (size_t)seg * L.seg_stride : nullptr) : A.init;
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      h[i] = zero4();
      if (init && own(i)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = init[sbase + state_at(i, j)];
      }
    }
    auto put_state = [&](int c) __attribute__((always_inline)) {   // H^T [column][row] as the A operand of H^T X^T
      if constexpr (OUT) {
        unsigned char* hs = set_of(c) + H_OFF;
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
          if (!own(i)) continue;
          if constexpr (BF) {
            const int off = state_piece<S::YROW>(16 * dvt + r, 2 * (rt0 + i) + (g >> 1)) + (g & 1) * 8;
            u32x2 a, b;
            uint32_t ha, la, hb, lb;
            split_pair_bf16(h[i][0], h[i][1], ha, la);
            split_pair_bf16(h[i][2], h[i][3], hb, lb);
            a = u32x2{ha, hb};
            b = u32x2{la, lb};
            *reinterpret_cast<u32x2*>(hs + off) = a;
            *reinterpret_cast<u32x2*>(hs + S::H_BYTES + off) = b;
          } else {
            const int off = state_piece<S::YROW>(16 * dvt + r, 4 * (rt0 + i) + g);
            *reinterpret_cast<f32x4*>(hs + off) = h[i];
          }
        }
      }
    };
    put_state(0);
    lds_barrier();   // the first decay factors are there
    lds_barrier();   // set 0 is filled
    float decay = 1.f;   // product of the chunks' decays
    auto chunk = [&](int c, const unsigned char* set) __attribute__((always_inline)) {
      const float* dec = dec_of(c);
      // A operand: the columns of Y this wave's row tiles are; B operand: the
      // terms of G(C, s) z_s for its column tile
      Frag zf[KBC][S::ZSETS], yf[KBC][TPW];
#pragma unroll
      for (int kb = 0; kb < KBC; ++kb) {
#pragma unroll
        for (int i = 0; i < TPW; ++i) yf[kb][i] = col_frag<T, S::YROW>(set, 16 * min(rt0 + i, S::RH - 1), kb, g, r);
#pragma unroll
        for (int n = 0; n < S::ZSETS; ++n)
          zf[kb][n] = col_frag<T, S::ZROW>(set + ZS_OFF + n * S::Z_BYTES, 16 * dvt, kb, g, r);
      }
      const float end = dec[2 * C + C - 1];
      decay *= end;
#pragma unroll
      for (int i = 0; i < TPW; ++i) h[i] *= end;
#pragma unroll
      for (int kb = 0; kb < KBC; ++kb)
#pragma unroll
        for (int n = S::ZSETS - 1; n >= 0; --n)
#pragma unroll
          for (int i = 0; i < TPW; ++i) h[i] = mma<T>(h[i], yf[kb][i], zf[kb][n]);
      put_state(c + 1);
      lds_barrier();
    };
    for (int c = 0; c < nch; c += 2) {
      chunk(c, set_of(0));
      if (c + 1 >= nch) break;
      chunk(c + 1, set_of(1));
    }
    // the final state (of the last segment), or this segment's own state
    float* fin = OUT ? (seg == L.nseg - 1 ? A.fin : nullptr) : A.seg_out + (size_t)seg * L.seg_stride;
    if (fin) {
      // dh0 = a_1 R_1: the first row's own decay, which a reversed sweep has not applied
      float scale = 1.f;
      if (A.reverse && len > 0 && OUT) {
        const float x = to_f32(*gp) * kLog2E;
        scale = __builtin_amdgcn_exp2f(x < kDecayFloor ? kDecayFloor : x);
      }
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        if (!own(i)) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) fin[sbase + state_at(i, j)] = h[i][j] * scale;
      }
    }
    if (!OUT && slice == 0 && sw == 0 && lane == 0) A.seg_decay[(size_t)seg * L.units * L.group + bh] = decay;
  } else {
    // ============================================================ copy waves
    const int cw = wave - (OUT ? 8 : 4), ct = tid - (OUT ? 512 : 256);
    const __amdgpu_buffer_rsrc_t yr = rows_rsrc(A.y, A.y_shared, D1, E);
    const __amdgpu_buffer_rsrc_t zr = rows_rsrc(A.z, A.z_shared, A.d2, E);
    const __amdgpu_buffer_rsrc_t gr = make_rsrc(gp, (uint32_t)((L.head_decay ? 1 : len) * E));
    struct Regs {
      Frag y[S::NY], z[S::NZ];
      T g;   // as stored: widened when placed, so that loading does not wait
    };
    auto load = [&](Regs& d, int c) __attribute__((always_inline)) {
      {   // the decay of the chunk's row `lane`: reversed row j carries that of the row after it
        const int j = row0 + C * c + lane, at = A.reverse ? len - j : j;
        const int off = j < len && at < len ? (L.head_decay ? 0 : at * E) : 0x7FFFFFF0;   // out of range: 0
        if constexpr (BF) d.g.bits = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(gr, off, 0, 0);
        else d.g = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(gr, off, 0, 0));
      }
#pragma unroll
      for (int j = 0; j < S::NY; ++j) {
        const int p = ct + 256 * j;
        const int row = first + dir * (C * c + p / S::YPR);
        d.y[j].w = __builtin_amdgcn_raw_buffer_load_b128(yr, row * D1 * E + (p % S::YPR) * 16, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < S::NZ; ++j) {
        const int p = ct + 256 * j;
        const int row = first + dir * (C * c + p / S::ZPR);
        d.z[j].w = __builtin_amdgcn_raw_buffer_load_b128(zr, (row * A.d2 + slice * DS) * E + (p % S::ZPR) * 16, 0, 0);
      }
    };
    auto factors = [&](const Regs& d, int c) __attribute__((always_inline)) {
      if (cw == 0) {
        float x = to_f32(d.g) * kLog2E;
        x = x < kDecayFloor ? kDecayFloor : x;   // keeps NaN
        const float whole = rintf(x * 64.f) * (1.f / 64.f);
        const float ch = wave_prefix(whole), cl = wave_prefix(x - whole);
        const float th = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ch), 63));
        const float tl = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, cl), 63));
        float* dec = dec_of(c);
        dec[lane] = ch;
        dec[C + lane] = cl;
        dec[2 * C + lane] = __builtin_amdgcn_exp2f(ch + cl);
        dec[3 * C + lane] = __builtin_amdgcn_exp2f((th - ch) + (tl - cl));
        dec[4 * C + lane] = __builtin_amdgcn_exp2f((row_last(ch) - ch) + (row_last(cl) - cl));
      }
    };
    auto place = [&](const Regs& d, int c) __attribute__((always_inline)) {
      unsigned char* set = set_of(c);
      const float* dec = dec_of(c);
#pragma unroll
      for (int j = 0; j < S::NY; ++j) {
        const int p = ct + 256 * j;
        if (C * S::YPR % 256 == 0 || p < C * S::YPR)
          store_frag(set + lds_piece<S::YROW>(p / S::YPR, p % S::YPR), d.y[j]);
      }
#pragma unroll
      for (int j = 0; j < S::NZ; ++j) {
        const int p = ct + 256 * j;
        if (C * S::ZPR % 256 == 0 || p < C * S::ZPR) {
          const int off = lds_piece<S::ZROW>(p / S::ZPR, p % S::ZPR);
          store_frag(set + Z_OFF + off, d.z[j]);
          const float wt = dec[3 * C + p / S::ZPR];   // G(C, row)
          if constexpr (BF) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              v[e] = wt * ((e & 1) ? bf16_hi_half(d.z[j].w[e >> 1]) : bf16_lo_half(d.z[j].w[e >> 1]));
            Frag t[3];
            split3_bf16(v, t[0], t[1], t[2]);
#pragma unroll
            for (int n = 0; n < S::ZSETS; ++n) store_frag(set + ZS_OFF + n * S::Z_BYTES + off, t[n]);
          } else {
            store_frag(set + ZS_OFF + off, frag_from_acc_f32(__builtin_bit_cast(f32x4, d.z[j].w) * wt));
          }
        }
      }
    };
    if constexpr (S::D1P != D1) {
      // half K blocks: the columns behind D1 are zero for good
      for (int p = ct; p < 2 * C * 2; p += 256) {
        unsigned char* set = set_of(p & 1);
        const int row = (p >> 1) >> 1, piece = 2 + ((p >> 1) & 1);
        store_frag(set + lds_piece<S::YROW>(row, piece), Frag{u32x4{0, 0, 0, 0}});
        if (OUT && row < DS) {
          store_frag(set + H_OFF + state_piece<S::YROW>(row, piece), Frag{u32x4{0, 0, 0, 0}});
          store_frag(set + H_OFF + S::H_BYTES + state_piece<S::YROW>(row, piece), Frag{u32x4{0, 0, 0, 0}});
        }
      }
    }
    // Chunk x is loaded into register set x % 2 two iterations before it is
    // placed.  Loads and copies run on past the last chunk (the last one again,
    // into sets nobody reads): a conditional load would make every wait for an
    // older one wait for all loads in flight.
    // The decay factors are a chunk ahead of the copies that use them.
    Regs r0, r1;
    load(r0, 0);
    load(r1, min(1, last));
    factors(r0, 0);
    lds_barrier();   // the first decay factors are there
    place(r0, 0);
    factors(r1, 1);
    load(r0, min(2, last));
    lds_barrier();   // set 0 is filled
    for (int c = 0; c < nch; c += 2) {
      place(r1, c + 1);
      factors(r0, c + 2);
      load(r1, min(c + 3, last));
      lds_barrier();
      if (c + 1 >= nch) break;
      place(r0, c + 2);
      factors(r1, c + 3);
      load(r0, min(c + 4, last));
      lds_barrier();
    }
  }
}

// Segment states, in place: segment i holds its own state (from zero) on entry
// and its start on return, start[0] = init, start[i + 1] = decay_i start[i] +
// own_i.  One thread per four state elements of one (batch, head).
__global__ __launch_bounds__(256) void segment_scan_kernel(float* states, const float* decay, const float* init,
                                                           int nseg, int heads, long long elems, long long seg_stride) {
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= heads * elems) return;
  const int bh = (int)(i / elems);
  f32x4 h = init ? *reinterpret_cast<const f32x4*>(init + i) : zero4();
  for (int s = 0; s < nseg; ++s) {
    f32x4* p = reinterpret_cast<f32x4*>(states + s * seg_stride + i);
    if (s + 1 < nseg) {
      const f32x4 mine = *p;
      const float d = decay[(size_t)s * heads + bh];
      *p = h;
      h = d * h + mine;
    } else {
      *p = h;
    }
  }
}

template <typename T, int D1, int DS, bool OUT, bool EXACT>
hipError_t launch_sweep_t(const SweepLaunch& L, hipStream_t stream) {
  const long long wgs = (long long)L.units * L.parts;
  if (wgs == 0) return hipSuccess;
  hipLaunchKernelGGL((sweep_kernel<T, D1, DS, OUT, EXACT>), dim3((unsigned)wgs), dim3(OUT ? 768 : 512), 0, stream, L);
  return hipGetLastError();
}

template <typename T, int D1, int DS>
hipError_t launch_sweep_o(const SweepLaunch& L, bool out, hipStream_t stream) {
  if (!out) return launch_sweep_t<T, D1, DS, false, true>(L, stream);
  // (fp32 products have one term: one instantiation)
  return L.exact_state || sizeof(T) == 4 ? launch_sweep_t<T, D1, DS, true, true>(L, stream)
                                         : launch_sweep_t<T, D1, DS, true, sizeof(T) == 4>(L, stream);
}

template <typename T, int D1>
hipError_t launch_sweep_d(const SweepLaunch& L, int ds, bool out, hipStream_t stream) {
  return ds == 32 ? launch_sweep_o<T, D1, 32>(L, out, stream) : launch_sweep_o<T, D1, 16>(L, out, stream);
}

template <typename T>
hipError_t launch_sweep_e(const SweepLaunch& L, int d1, int ds, bool out, hipStream_t stream) {
  switch (d1) {
    case 16: return launch_sweep_d<T, 16>(L, ds, out, stream);
    case 32: return launch_sweep_d<T, 32>(L, ds, out, stream);
    case 64: return launch_sweep_d<T, 64>(L, ds, out, stream);
    case 128: return launch_sweep_d<T, 128>(L, ds, out, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// ---------------------------------------------------------------- decay gradient
// dg_t = a_t <R_t, H_{t-1}> is everything that passes gate t: the pairs of a
// key before t and a query from t on, with the initial state among the keys and
// dhT among the queries.  With a_u = q_u . dq_u (every pair ending at query u)
// and b_u = k_u . dk_u (every pair starting at key u)
//   dg_t = <dhT, H_T> + sum_{u >= t} (a_u - b_u),
// a running sum from the sequence's end.  The sweeps leave the parts of a and b
// per slice, taken from their unrounded outputs; the sum runs in fp64.
// One workgroup per (batch, head), four rows per thread.
constexpr int kDgThreads = 1024;

__device__ __forceinline__ double wave_prefix_f64(double x, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  return x;
}

template <typename T>
__global__ __launch_bounds__(kDgThreads) void decay_grad_kernel(const float* dotq, const float* dotk, int slices,
                                                                const float* dhT, const float* hT, int elems,
                                                                const int* lens, int rows, int heads, int nbh, T* dg,
                                                                double* head_sum) {
  __shared__ double s_wave[kDgThreads / 64], s_total;
  const int bh = blockIdx.x, tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int len = lens ? min(max(lens[bh / heads], 0), rows) : rows;
  // sum over the workgroup, and the exclusive prefix of this thread
  auto scan = [&](double x, double& total) __attribute__((always_inline)) {
    const double inc = wave_prefix_f64(x, lane);
    if (lane == 63) s_wave[wave] = inc;
    __syncthreads();
    if (wave == 0) {
      const double w = lane < kDgThreads / 64 ? s_wave[lane] : 0.0;
      const double winc = wave_prefix_f64(w, lane);
      if (lane < kDgThreads / 64) s_wave[lane] = winc - w;
      if (lane == 63) s_total = winc;
    }
    __syncthreads();
    const double before = s_wave[wave] + (inc - x);
    total = s_total;
    __syncthreads();
    return before;
  };
  double carry = 0.0;
  if (dhT) {
    double x = 0.0;
    for (int i = tid; i < elems; i += kDgThreads) x += (double)dhT[(size_t)bh * elems + i] * hT[(size_t)bh * elems + i];
    scan(x, carry);
  }
  double sum = 0.0;
  for (int base = 0; base < len; base += 4 * kDgThreads) {   // counted from the end
    double d[4], mine = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = len - 1 - (base + 4 * tid + j);
      double x = 0.0;
      if (row >= 0)
        for (int s = 0; s < slices; ++s) {
          const size_t at = ((size_t)s * nbh + bh) * rows + row;
          x += (double)dotq[at] - (double)dotk[at];
        }
      mine += x;
      d[j] = mine;
    }
    double total;
    const double before = carry + scan(mine, total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = len - 1 - (base + 4 * tid + j);
      if (row < 0) continue;
      if (head_sum) sum += before + d[j];
      else dg[(size_t)bh * rows + row] = from_f32<T>((float)(before + d[j]));
    }
    carry += total;
  }
  if (head_sum) {
    double total;
    scan(sum, total);
    if (tid == 0) head_sum[bh] = total;
  }
}

template <typename T>
__global__ __launch_bounds__(64) void head_decay_grad_kernel(const double* head_sum, int B, int H, T* dg) {
  const int h = blockIdx.x * 64 + threadIdx.x;
  if (h >= H) return;
  double x = 0.0;
  for (int b = 0; b < B; ++b) x += head_sum[(size_t)b * H + h];
  dg[h] = from_f32<T>((float)x);
}

// Gradients of a query or key shared by `group` heads: the sum of the heads'
// fp32 parts [units, group, rows, d], rounded once.  Four elements per thread.
template <typename T>
__global__ __launch_bounds__(256) void fold_heads_kernel(const float* parts, int units, int group, int rows, int d,
                                                         const int* lens, int units_per_batch, T* out) {
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
// of q_i H_i go through LDS.
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
  const float a = expf(to_f32(gate[head_decay ? st % heads : st]));
  __syncthreads();
  f32x4 acc = zero4();
#pragma unroll
  for (int j = 0; j < ITER; ++j) {
    const int row = rg + j * RPI;
    if (row < DK) {
      const f32x4 hn = a * h[j] + s_k[row] * vv;
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
  int dvs = a.dv;
  while (dvs > 16 && states * (a.dv / dvs) < 256) dvs /= 2;   // few states: their columns over more CUs
  return a.dtype == 1 ? la_decode_dk<bf16_t>(a, dvs) : la_decode_dk<float>(a, dvs);
}

// ---------------------------------------------------------------- host side

static hipError_t launch_sweep(const SweepLaunch& L, int dtype, int d1, int ds, bool out, hipStream_t stream) {
  return dtype == 1 ? launch_sweep_e<bf16_t>(L, d1, ds, out, stream) : launch_sweep_e<float>(L, d1, ds, out, stream);
}

static int slice_width(int d2) { return d2 >= 32 ? 32 : 16; }

// Rows of a segment: one segment when the (batch, head, slice) workgroups of
// one sweep fill the CUs, else enough segments to give every CU one, of at
// least eight chunks each (every further segment re-reads its rows once more,
// for its own state).
static int segment_rows(long long wgs, int T) {
  constexpr int kCUs = 256, kMinChunks = 8;
  const int nch = (T + C - 1) / C;
  long long nseg = wgs > 0 ? kCUs / wgs : 1;
  if (nseg > nch / kMinChunks) nseg = nch / kMinChunks;
  if (nseg < 1) nseg = 1;
  return (int)((nch + nseg - 1) / nseg) * C;
}
static int segment_count(int T, int rows) { return T <= rows ? 1 : (T + rows - 1) / rows; }

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// workspace of the forward: the segments' states and decays
struct FwdPlan {
  int seg_rows, nseg;
  size_t states, decay, bytes;
};
static FwdPlan fwd_plan(int B, int H, int T, int dk, int dv) {
  FwdPlan p;
  const size_t bh = (size_t)B * H;
  p.seg_rows = segment_rows((long long)bh * (dv / slice_width(dv)), T);
  p.nseg = segment_count(T, p.seg_rows);
  p.states = 0;
  p.decay = p.nseg > 1 ? up256((size_t)p.nseg * bh * dk * dv * 4) : 0;
  p.bytes = p.nseg > 1 ? p.decay + up256((size_t)p.nseg * bh * 4) : 0;
  return p;
}
size_t linattn_fwd_workspace_bytes(int B, int H, int T, int dk, int dv) { return fwd_plan(B, H, T, dk, dv).bytes; }

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

// states of the segments of one direction: own states, then their starts
static hipError_t segment_starts(const LinAttnArgs& a, bool reverse, int seg_rows, int nseg, float* states, float* decay,
                                 const float* init) {
  SweepLaunch L = sweep_base(a);
  const int ds = slice_width(a.dv);
  const size_t bh = (size_t)a.B * a.H, elems = (size_t)a.dk * a.dv;
  L.seg_rows = seg_rows;
  L.nseg = nseg;
  L.seg_stride = (long long)(bh * elems);
  L.nroles = 1;
  SweepRole& R = L.role[0];
  R.y = reverse ? a.q : a.k;
  R.y_shared = 1;
  R.z = reverse ? a.dout : a.v;
  R.reverse = reverse;
  R.d2 = a.dv;
  R.seg_out = states;
  R.seg_decay = decay;
  R.parts = L.parts = (nseg - 1) * L.group * (a.dv / ds);
  hipError_t e = launch_sweep(L, a.dtype, a.dk, ds, false, a.stream);
  if (e != hipSuccess) return e;
  const long long threads = (long long)(bh * elems / 4);
  hipLaunchKernelGGL(segment_scan_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, a.stream, states, decay,
                     init, nseg, (int)bh, (long long)elems, L.seg_stride);
  return hipGetLastError();
}

hipError_t launch_linattn_fwd(const LinAttnArgs& a) {
  const FwdPlan p = fwd_plan(a.B, a.H, a.T, a.dk, a.dv);
  unsigned char* ws = (unsigned char*)a.workspace;
  float* states = (float*)(ws + p.states);
  if (p.nseg > 1) {
    hipError_t e = segment_starts(a, false, p.seg_rows, p.nseg, states, (float*)(ws + p.decay), a.h0);
    if (e != hipSuccess) return e;
  }
  SweepLaunch L = sweep_base(a);
  const int ds = slice_width(a.dv);
  L.seg_rows = p.seg_rows;
  L.nseg = p.nseg;
  L.seg_stride = (long long)a.B * a.H * a.dk * a.dv;
  L.nroles = 1;
  SweepRole& R = L.role[0];
  R.x = a.q;
  R.y = a.k;
  R.x_shared = R.y_shared = 1;
  R.z = a.v;
  R.d2 = a.dv;
  R.out = a.o;
  R.init = a.h0;
  R.fin = a.hT;
  R.seg_states = states;
  L.exact_state = a.hT != nullptr;
  R.parts = L.parts = p.nseg * L.group * (a.dv / ds);
  return launch_sweep(L, a.dtype, a.dk, ds, true, a.stream);
}

// workspace of the backward: dots of queries and keys with their gradients,
// the final state, segment states of both directions, and the heads' parts of
// shared gradients
struct BwdPlan {
  int seg_rows, nseg;
  size_t dotq, dotk, hT, head_sum, states, rstates, decay, dq, dk, bytes;
};
static BwdPlan bwd_plan(int B, int H, int Hk, int T, int dk, int dv) {
  BwdPlan p;
  const size_t bh = (size_t)B * H, elems = (size_t)dk * dv;
  const int sk = dk / slice_width(dk), sv = dv / slice_width(dv);
  p.seg_rows = segment_rows((long long)bh * (2 * sk + sv), T);
  p.nseg = segment_count(T, p.seg_rows);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  p.dotq = take((size_t)sk * bh * T * 4);
  p.dotk = take((size_t)sk * bh * T * 4);
  p.hT = take(bh * elems * 4);
  p.head_sum = take(bh * 8);
  p.states = take(p.nseg > 1 ? (size_t)p.nseg * bh * elems * 4 : 0);
  p.rstates = take(p.nseg > 1 ? (size_t)p.nseg * bh * elems * 4 : 0);
  p.decay = take(p.nseg > 1 ? (size_t)p.nseg * bh * 4 : 0);
  const bool grouped = H != Hk;
  p.dq = take(grouped ? bh * T * dk * 4 : 0);
  p.dk = take(grouped ? bh * T * dk * 4 : 0);
  p.bytes = at;
  return p;
}
size_t linattn_bwd_workspace_bytes(int B, int H, int Hk, int T, int dk, int dv) {
  return bwd_plan(B, H, Hk, T, dk, dv).bytes;
}

template <typename T>
static hipError_t launch_bwd_tail(const LinAttnArgs& a, const BwdPlan& p, unsigned char* ws) {
  const int bh = a.B * a.H, slices = a.dk / slice_width(a.dk);
  double* sums = a.head_decay ? (double*)(ws + p.head_sum) : nullptr;
  hipError_t e = hipSuccess;
  if (bh > 0)
    hipLaunchKernelGGL((decay_grad_kernel<T>), dim3(bh), dim3(kDgThreads), 0, a.stream, (const float*)(ws + p.dotq),
                       (const float*)(ws + p.dotk), slices, a.dhT, (const float*)(ws + p.hT), a.dk * a.dv, a.lens, a.T,
                       a.H, bh, (T*)a.dg, sums);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.head_decay) {
    hipLaunchKernelGGL((head_decay_grad_kernel<T>), dim3((a.H + 63) / 64), dim3(64), 0, a.stream, sums, a.B, a.H,
                       (T*)a.dg);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (a.H != a.Hk && bh > 0 && a.T > 0) {
    const int units = a.B * a.Hk;
    const long long threads = (long long)units * a.T * a.dk / 4;
    for (int i = 0; i < 2; ++i) {
      hipLaunchKernelGGL((fold_heads_kernel<T>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, a.stream,
                         (const float*)(ws + (i ? p.dk : p.dq)), units, a.H / a.Hk, a.T, a.dk, a.lens, a.Hk,
                         (T*)(i ? a.dk_out : a.dq));
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

hipError_t launch_linattn_bwd(const LinAttnArgs& a) {
  const BwdPlan p = bwd_plan(a.B, a.H, a.Hk, a.T, a.dk, a.dv);
  unsigned char* ws = (unsigned char*)a.workspace;
  float *states = (float*)(ws + p.states), *rstates = (float*)(ws + p.rstates);
  hipError_t e;
  if (p.nseg > 1) {
    float* decay = (float*)(ws + p.decay);
    if ((e = segment_starts(a, false, p.seg_rows, p.nseg, states, decay, a.h0)) != hipSuccess) return e;
    if ((e = segment_starts(a, true, p.seg_rows, p.nseg, rstates, decay, a.dhT)) != hipSuccess) return e;
  }
  const bool grouped = a.H != a.Hk;
  const int dsk = slice_width(a.dk), dsv = slice_width(a.dv);
  SweepRole dv = {}, dk = {}, dq = {};
  dv.x = a.k;
  dv.y = a.q;
  dv.x_shared = dv.y_shared = 1;
  dv.z = a.dout;
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
  dq.fin = a.dhT ? (float*)(ws + p.hT) : nullptr;   // <dhT, H_T> of the decay gradient
  dq.seg_states = states;
  SweepLaunch L = sweep_base(a);
  L.seg_rows = p.seg_rows;
  L.nseg = p.nseg;
  L.seg_stride = (long long)a.B * a.H * a.dk * a.dv;
  L.exact_state = a.dh0 || a.dhT;
  const int per = p.nseg * L.group;
  dv.parts = per * (a.dv / dsv);
  dk.parts = dq.parts = per * (a.dk / dsk);
  // one launch where the sweeps have the same widths, else the two that
  // contract over dv apart from the one over dk
  if (a.dk == a.dv) {
    L.role[0] = dv;
    L.role[1] = dk;
    L.role[2] = dq;
    L.nroles = 3;
    L.parts = dv.parts + dk.parts + dq.parts;
    if ((e = launch_sweep(L, a.dtype, a.dk, dsk, true, a.stream)) != hipSuccess) return e;
  } else {
    L.role[0] = dv;
    L.nroles = 1;
    L.parts = dv.parts;
    if ((e = launch_sweep(L, a.dtype, a.dk, dsv, true, a.stream)) != hipSuccess) return e;
    L.role[0] = dk;
    L.role[1] = dq;
    L.nroles = 2;
    L.parts = dk.parts + dq.parts;
    if ((e = launch_sweep(L, a.dtype, a.dv, dsk, true, a.stream)) != hipSuccess) return e;
  }
  return a.dtype == 1 ? launch_bwd_tail<bf16_t>(a, p, ws) : launch_bwd_tail<float>(a, p, ws);
}

}  // namespace ckda
