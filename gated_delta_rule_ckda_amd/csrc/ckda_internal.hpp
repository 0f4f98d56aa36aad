// ckda_internal.hpp -- host-side launch descriptors shared between the C ABI
// layer (argument checking, dispatch) and the kernel translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "ckda.h"

namespace ckda {

// Launch flag beside the public CKDA_FUSE_* / CKDA_GATE_SCALAR bits: two
// delta-rule sub-steps per token (DeltaProduct_2; rows of k, v, beta are
// sub-steps, rows of q, o and of a scalar alpha are tokens).
constexpr int kProd2 = 1 << 16;

struct DecodeArgs {
  const void *q, *k, *v, *alpha, *beta;
  float* H_inout;
  void* o;
  int N, H, dk, dv, dtype;
  int flags;   // CKDA_FUSE_* prologue steps (0: inputs used as given)
  hipStream_t stream;
  const int* gidx = nullptr;   // [H][dk] retained channel indices into rows of dk_in (NULL: no gather)
  int dk_in = 0;
};

struct ChunkArgs {
  const void *q, *k, *v, *alpha, *beta;
  const float* h0;
  void* o;
  float* hT;
  int B, H, T, dk, dv, chunk, dtype;
  int flags;   // CKDA_FUSE_* prologue steps (0: inputs used as given)
  void* workspace;
  hipStream_t stream;
  hipEvent_t ev[3];   // recorded before the Gram kernel, between the kernels, after the state kernel (if set)
  const int* gidx = nullptr;   // [H][dk] retained channel indices into rows of dk_in (NULL: no gather)
  int dk_in = 0;
};

// Layout of the per-chunk records the Gram kernel writes and the state-pass
// kernel reads (byte offsets inside one chunk's record).
struct ChunkRecord {
  size_t t_off, m_off, bytes;
};
ChunkRecord chunk_record_layout(int dk, int chunk, int dtype);

struct BwdArgs {
  const void *q, *k, *v, *alpha, *beta;
  const float* h0;
  const void* dout;
  const float* dhT;
  float *gq, *gk, *gv, *galpha, *gbeta, *gh0;   // gradients of q, k, v, alpha, beta, h0
  int B, H, T, dk, dv, dtype;
  void* workspace;
  hipStream_t stream;
};
// floats of backward workspace (per-chunk records, chunk-start states and
// state gradients), 0 for an unsupported dk
size_t chunk_bwd_workspace_floats(int B, int H, int T, int dk, int dv);
hipError_t launch_chunk_bwd(const BwdArgs& a);
// the backward through the per-token prologue (prologue_bwd.hip); flags as
// CKDA_FUSE_* | CKDA_GATE_SCALAR, nonzero
size_t prologue_bwd_workspace_floats(int B, int H, int T, int dk, int dv, int flags);
hipError_t launch_prologue_bwd(const BwdArgs& a, int flags);
// the DeltaProduct_2 backward (dp2_bwd.hip): k, v, beta, dk, dv, dbeta hold 2 T
// sub-steps; alpha (or NULL: ungated) and dalpha are [B, H, T]
size_t dp2_bwd_workspace_bytes(int B, int H, int T, int dk, int dv, int dtype);
hipError_t launch_dp2_bwd(const BwdArgs& a);

hipError_t launch_decode(const DecodeArgs& a);
hipError_t launch_chunk_fwd(const ChunkArgs& a);

// ---- linear attention with a decay for each head (linattn.hip)
constexpr int kLaChunk = 64;   // rows of a chunk

struct LinAttnArgs {
  const void *q, *k, *v, *g;
  const float* h0;
  const void* dout;          // backward: dL/do, dL/dH_T, gradients
  const float* dhT;
  void* o;                   // forward: outputs, final state
  float* hT;
  void *dq, *dk_out, *dv_out, *dg;
  float* dh0;
  const int* lens;           // [B] or NULL
  int B, H, Hk, T, dk, dv, dtype, head_decay;
  void* workspace;
  hipStream_t stream;
};
struct LinAttnDecodeArgs {
  const void *q, *k, *v, *g;
  float* H_inout;
  void* o;
  int N, H, Hk, dk, dv, dtype, head_decay;
  hipStream_t stream;
};

// One sweep: out_t = S_t^T x_t with S_t = a_t S_{t-1} + y_t z_t^T, S [d1, d2].
// An operand that is `shared` has one head for the group's heads.
struct SweepRole {
  const void *x, *y, *z;
  const void* w;             // dot[part][slice][bh][row] = w_row . out_row over the slice (or NULL), of
  float* dot;                // the rows before the row's chunk (part 0) and of those in it before the row (1)
  void* out;
  const float* init;         // first state (or NULL: zero)
  float* fin;                // last state (or NULL)
  float* seg_states;         // start state of every sub-segment (with more than one segment)
  float* seg_out;            // own-state launches: the sub-segments' own states and decays (two floats each)
  float2* seg_decay;
  int x_shared, y_shared, z_shared, w_shared;
  int d1, d2;
  int reverse;               // from the last row to the first
  int turned;                // init, fin and segment states are stored [d2, d1]
  int out_f32;               // out is fp32
  int drop_end;              // states without the rows of a sequence's last chunk (its decay applied)
  int parts;                 // workgroups per unit and segment: heads of the group x slices
};
struct SweepLaunch {
  SweepRole role[3];
  const void* g;
  const int* lens;
  long long seg_stride;      // floats between two segments' states
  int nroles, units, group, heads, rows, parts, seg_rows, nseg, seg_subs, head_decay;
  int exact_state;           // state products with three bf16 terms (a state is returned), else two
};

size_t linattn_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, int dtype);
size_t linattn_bwd_workspace_bytes(int B, int H, int Hk, int T, int dk, int dv, int dtype);
bool linattn_fits_grid(int B, int H, int Hk, int T, int dk, int dv, int dtype, bool backward);
hipError_t launch_linattn_fwd(const LinAttnArgs& a);
hipError_t launch_linattn_bwd(const LinAttnArgs& a);
hipError_t launch_linattn_decode(const LinAttnDecodeArgs& a);

// ---- norm of the attention output by head, with an output gate (head_norm.hip)
struct HeadNormArgs {
  const void *x, *z, *dy;
  const float *w, *b;
  void *y, *dx, *dz;
  float *dw, *db;
  int B, H, T, D, wheads, dtype, flags;
  float eps;
  void* workspace;
  hipStream_t stream;
};
size_t head_norm_bwd_workspace_bytes(int B, int H, int T, int D, int wheads, int dtype);
hipError_t launch_head_norm_fwd(const HeadNormArgs& a);
hipError_t launch_head_norm_bwd(const HeadNormArgs& a);

// ---- sums over parts, in a fixed order (part_sums.hip)
// out[i] = sum over p of part[p * stride + i], for columns that lie side by side
// in a part: up to three outputs (NULL: skipped) of cols[] columns each.
struct PartSums {
  const float* part;
  int nparts;
  size_t stride;
  float* out[3];
  size_t cols[3];
};
hipError_t launch_part_sums(const PartSums& s, hipStream_t stream);

// ---- short causal convolution (short_conv.hip)
struct ShortConvArgs {
  const void* x;
  const float *w, *b;
  const void* s0;            // inputs before the first row (or NULL)
  const int* lens;           // [B] or NULL
  void *y, *sT;              // forward: outputs, last inputs (or NULL)
  const void *dy, *dsT;      // backward
  void* dx;
  float *dw, *db;
  void* ds0;
  void* state;               // decode: state in place
  int B, T, C, H, K, ldx, dtype, silu, pad_zero;
  void* workspace;
  hipStream_t stream;
};
size_t short_conv_bwd_workspace_bytes(int B, int T, int C, int K);
bool short_conv_fits_grid(int B, int T, int C, int H);
hipError_t launch_short_conv_fwd(const ShortConvArgs& a);
hipError_t launch_short_conv_bwd(const ShortConvArgs& a);
hipError_t launch_short_conv_decode(const ShortConvArgs& a);

// ---- selective scan (selective_scan.hip)
struct SelScanArgs {
  const void *x, *dt;
  const float* A;
  const void *Bm, *Cm;
  const float* D;
  const void* z;
  const float* dt_bias;
  const float* h0;
  const int* lens;           // [B] or NULL
  void* y;
  float* hT;
  const void* dy;            // backward
  const float* dhT;
  void *dx, *ddt, *dBm, *dCm, *dz;
  float *dA, *dD, *dbias, *dh0;
  float* H_inout;            // decode: state in place
  int B, T, C, G, N, ldbc, ldz, dtype, softplus, pad_zero;
  void* workspace;
  hipStream_t stream;
};
size_t scan_fwd_workspace_bytes(int B, int T, int C, int G, int N);
size_t scan_bwd_workspace_bytes(int B, int T, int C, int G, int N);
bool scan_fits_grid(int B, int T, int C, int G, int N);
hipError_t launch_scan_fwd(const SelScanArgs& a);
hipError_t launch_scan_bwd(const SelScanArgs& a);
hipError_t launch_scan_decode(const SelScanArgs& a);

// ---- norm with the residual's addition (add_norm.hip)
struct AddNormArgs {
  const void *x, *res;
  const float* w;
  void *y, *q;
  float* scales;
  void* sum;                 // forward: stored sum (or NULL); backward: its input
  const void *dy, *dsum;     // backward
  void *dx, *dres;
  float* dw;
  int R, D, group, dtype, res_dtype;
  float eps;
  void* workspace;
  hipStream_t stream;
};
size_t add_norm_bwd_workspace_bytes(int R, int D, int dtype);
hipError_t launch_add_norm_fwd(const AddNormArgs& a);
hipError_t launch_add_norm_bwd(const AddNormArgs& a);

// Size of the fixed device scratch of ckda_chunk_fwd_noalloc (noalloc.hip),
// and its device address on the current device (looked up on first use).
constexpr size_t kNoallocScratchBytes = (size_t)64 << 20;
hipError_t noalloc_scratch(void** ptr);

}  // namespace ckda
