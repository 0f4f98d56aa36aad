// linattn_api.cpp -- the C ABI of the linear attention with a decay for each
// head and of the head norm (include/ckda.h): argument, aliasing and workspace
// checks, dispatch and error reporting.  As in ckda_api.cpp nothing here
// touches device memory and every check runs before a launch.
#include "ckda_checks.hpp"
#include "ckda_internal.hpp"

using namespace ckda;

extern "C" {

// ---------------------------------------------------------------- linear attention

// sizes common to the linear attention's entry points; rows = T (decode: 1)
static int linattn_sizes(const char* fn, int B, int H, int Hk, int T, int dk, int dv, int dtype, int flags) {
  if ((flags & ~CKDA_DECAY_HEAD) != 0)
    return fail(CKDA_ERR_FLAGS, "%s: flags 0x%x has bits outside CKDA_DECAY_HEAD (0x%x)", fn, flags, CKDA_DECAY_HEAD);
  if (B < 0 || H < 0 || T < 0) return fail(CKDA_ERR_DIM, "%s: negative size (B=%d H=%d T=%d)", fn, B, H, T);
  if (H > 0 && (Hk < 1 || H % Hk != 0)) return fail(CKDA_ERR_DIM, "%s: Hk=%d does not divide H=%d", fn, Hk, H);
  if (!supported_dtype(dtype)) return fail(CKDA_ERR_UNSUPPORTED, "%s: dtype %d is not F32(0) or BF16(1)", fn, dtype);
  if (!supported_dim(dk) || !supported_dim(dv))
    return fail(CKDA_ERR_UNSUPPORTED, "%s: dk=%d dv=%d (supported: 16, 32, 64, 128)", fn, dk, dv);
  return CKDA_OK;
}

// row offsets inside one head are 32-bit byte offsets, up to two chunks past the end
static bool linattn_rows_fit(int T, int dk, int dv, size_t es) {
  return ((size_t)T + 2 * ckda::kLaChunk) * (dk > dv ? dk : dv) * es <= (size_t)INT32_MAX;
}

// heads and rows whose products the host's arithmetic holds (wider calls are refused)
static bool linattn_planned(int B, int H, int T, int dk, int dv, size_t es) {
  return (size_t)B * H * 24 <= (size_t)INT32_MAX && linattn_rows_fit(T, dk, dv, es);
}

static int check_workspace(const char* fn, const void* workspace, size_t have, size_t need) {
  if (!workspace) return fail(CKDA_ERR_WORKSPACE, "%s: workspace is NULL", fn);
  if (have < need) return fail(CKDA_ERR_WORKSPACE, "%s: workspace of %zu bytes, need %zu", fn, have, need);
  if (((uintptr_t)workspace & 255u) != 0) return fail(CKDA_ERR_WORKSPACE, "%s: workspace not 256-byte aligned", fn);
  return CKDA_OK;
}

static int check_aligned(const char* fn, const Range* r, int n) {
  for (int i = 0; i < n; ++i)
    if (r[i].lo && misaligned((const void*)r[i].lo))
      return fail(CKDA_ERR_DIM, "%s: %s is not 16-byte aligned", fn, r[i].name);
  return CKDA_OK;
}

// no output overlaps an input or another output, and the workspace (among the
// inputs, or NULL) no input; `same` may equal `with` exactly
static int check_alias(const char* fn, const Range* in, int nin, const Range* out, int nout, const Range* ws,
                       const Range* same = nullptr, const Range* with = nullptr) {
  for (int j = 0; ws && j < nin; ++j)
    if (&in[j] != ws && overlap(*ws, in[j])) return fail(CKDA_ERR_ALIAS, "%s: workspace overlaps %s", fn, in[j].name);
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j) {
      if (&out[i] == same && &in[j] == with && same->lo == with->lo) continue;
      if (overlap(out[i], in[j])) return fail(CKDA_ERR_ALIAS, "%s: %s overlaps %s", fn, out[i].name, in[j].name);
    }
    for (int j = 0; j < nout; ++j)
      if (j != i && overlap(out[i], out[j]))
        return fail(CKDA_ERR_ALIAS, "%s: %s overlaps %s", fn, out[i].name, out[j].name);
  }
  return CKDA_OK;
}

// byte sizes of the linear attention's tensors
struct LinAttnSizes {
  size_t qk, v, g, states, lens;
};
static LinAttnSizes linattn_bytes(int B, int H, int Hk, int T, int dk, int dv, int dtype, int flags) {
  const size_t es = dtype_bytes(dtype), rows = (size_t)B * T;
  return LinAttnSizes{rows * Hk * dk * es, rows * H * dv * es, ((flags & CKDA_DECAY_HEAD) ? (size_t)H : rows * H) * es,
                      (size_t)B * H * dk * dv * 4, (size_t)B * 4};
}

size_t ckda_linattn_fwd_workspace_size(int B, int H, int T, int dk, int dv, int dtype) {
  if (B < 0 || H < 0 || T < 0) return 0;
  if (!supported_dim(dk) || !supported_dim(dv) || !supported_dtype(dtype)) return 0;
  if (!linattn_planned(B, H, T, dk, dv, dtype_bytes(dtype))) return 0;
  const size_t bytes = ckda::linattn_fwd_workspace_bytes(B, H, T, dk, dv, dtype);
  return bytes == 0 ? 256 : bytes;
}

int ckda_linattn_fwd(const void* q, const void* k, const void* v, const void* g, const float* h0, const int* lens,
                     void* o, float* hT, int B, int H, int Hk, int T, int dk, int dv, int dtype, int flags,
                     void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "ckda_linattn_fwd";
  int st = linattn_sizes(fn, B, H, Hk, T, dk, dv, dtype, flags);
  if (st != CKDA_OK) return st;
  const size_t BH = (size_t)B * H;
  if (BH == 0 || (T == 0 && !hT)) return ok();
  if (T > 0 && (!q || !k || !v || !g || !o)) return fail(CKDA_ERR_NULL, "%s: q, k, v, g and o are required", fn);
  if (BH * 24 > (size_t)INT32_MAX) return fail(CKDA_ERR_DIM, "%s: B*H too large", fn);
  if (!linattn_rows_fit(T, dk, dv, dtype_bytes(dtype)))
    return fail(CKDA_ERR_DIM, "%s: T=%d too long: one head's rows must stay below 2 GiB", fn, T);
  if (!ckda::linattn_fits_grid(B, H, Hk, T, dk, dv, dtype, false))
    return fail(CKDA_ERR_DIM, "%s: B*H exceeds the launch grid", fn);
  const size_t need = ckda_linattn_fwd_workspace_size(B, H, T, dk, dv, dtype);
  if (T > 0 && (st = check_workspace(fn, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const LinAttnSizes n = linattn_bytes(B, H, Hk, T, dk, dv, dtype, flags);
  const Range in[] = {range("q", q, n.qk), range("k", k, n.qk), range("v", v, n.v), range("g", g, g ? n.g : 0),
                      range("h0", h0, h0 ? n.states : 0), range("workspace", workspace, T ? need : 0),
                      range("lens", lens, lens ? n.lens : 0)};
  const Range out[] = {range("o", o, n.v), range("hT", hT, hT ? n.states : 0)};
  if ((st = check_aligned(fn, in, 6)) != CKDA_OK || (st = check_aligned(fn, out, 2)) != CKDA_OK) return st;
  if (lens && ((uintptr_t)lens & 3u) != 0) return fail(CKDA_ERR_DIM, "%s: lens is not 4-byte aligned", fn);
  if ((st = check_alias(fn, in, 7, out, 2, &in[5], &out[1], &in[4])) != CKDA_OK) return st;   // hT may be h0
  ckda::LinAttnArgs a = {};
  a.q = q, a.k = k, a.v = v, a.g = g, a.h0 = h0, a.o = o, a.hT = hT, a.lens = lens;
  a.B = B, a.H = H, a.Hk = Hk, a.T = T, a.dk = dk, a.dv = dv, a.dtype = dtype;
  a.head_decay = (flags & CKDA_DECAY_HEAD) != 0;
  a.workspace = workspace, a.stream = (hipStream_t)stream;
  const hipError_t e = ckda::launch_linattn_fwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

size_t ckda_linattn_bwd_workspace_size(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  if (B < 0 || H < 0 || T < 0 || (H > 0 && (Hk < 1 || H % Hk != 0))) return 0;
  if (!supported_dim(dk) || !supported_dim(dv) || !supported_dtype(dtype)) return 0;
  if (!linattn_planned(B, H, T, dk, dv, 4)) return 0;
  const size_t bytes = ckda::linattn_bwd_workspace_bytes(B, H, Hk, T, dk, dv, dtype);
  return bytes == 0 ? 256 : bytes;
}

int ckda_linattn_bwd(const void* q, const void* k, const void* v, const void* g, const float* h0, const int* lens,
                     const void* dout, const float* dhT, void* dq, void* dk_out, void* dv_out, void* dg, float* dh0,
                     int B, int H, int Hk, int T, int dk, int dv, int dtype, int flags, void* workspace,
                     size_t workspace_bytes, void* stream) {
  const char* fn = "ckda_linattn_bwd";
  int st = linattn_sizes(fn, B, H, Hk, T, dk, dv, dtype, flags);
  if (st != CKDA_OK) return st;
  const size_t BH = (size_t)B * H;
  // a constant decay has a gradient (zero) whatever the batch; everything else is empty without one
  const bool head = (flags & CKDA_DECAY_HEAD) != 0;
  if (H == 0 || (BH == 0 && !head)) return ok();
  if ((T > 0 && BH > 0 && (!q || !k || !v || !dout || !dq || !dk_out || !dv_out)) || ((T > 0 || head) && (!g || !dg)))
    return fail(CKDA_ERR_NULL, "%s: inputs, do and the gradients of q, k, v and g are required", fn);
  if (BH * 24 > (size_t)INT32_MAX) return fail(CKDA_ERR_DIM, "%s: B*H too large", fn);
  if (!linattn_rows_fit(T, dk, dv, 4))
    return fail(CKDA_ERR_DIM, "%s: T=%d too long: one head's rows must stay below 2 GiB (as fp32)", fn, T);
  if (!ckda::linattn_fits_grid(B, H, Hk, T, dk, dv, dtype, true))
    return fail(CKDA_ERR_DIM, "%s: sizes exceed the launch grid", fn);
  const size_t need = ckda_linattn_bwd_workspace_size(B, H, Hk, T, dk, dv, dtype);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const LinAttnSizes n = linattn_bytes(B, H, Hk, T, dk, dv, dtype, flags);
  const Range in[] = {range("q", q, n.qk), range("k", k, n.qk), range("v", v, n.v), range("g", g, g ? n.g : 0),
                      range("h0", h0, h0 ? n.states : 0), range("do", dout, n.v),
                      range("dhT", dhT, dhT ? n.states : 0), range("workspace", workspace, need),
                      range("lens", lens, lens ? n.lens : 0)};
  const Range out[] = {range("dq", dq, n.qk), range("dk", dk_out, n.qk), range("dv", dv_out, n.v),
                       range("dg", dg, dg ? n.g : 0), range("dh0", dh0, dh0 ? n.states : 0)};
  if ((st = check_aligned(fn, in, 8)) != CKDA_OK || (st = check_aligned(fn, out, 5)) != CKDA_OK) return st;
  if (lens && ((uintptr_t)lens & 3u) != 0) return fail(CKDA_ERR_DIM, "%s: lens is not 4-byte aligned", fn);
  if ((st = check_alias(fn, in, 9, out, 5, &in[7])) != CKDA_OK) return st;
  ckda::LinAttnArgs a = {};
  a.q = q, a.k = k, a.v = v, a.g = g, a.h0 = h0, a.lens = lens, a.dout = dout, a.dhT = dhT;
  a.dq = dq, a.dk_out = dk_out, a.dv_out = dv_out, a.dg = dg, a.dh0 = dh0;
  a.B = B, a.H = H, a.Hk = Hk, a.T = T, a.dk = dk, a.dv = dv, a.dtype = dtype;
  a.head_decay = head;
  a.workspace = workspace, a.stream = (hipStream_t)stream;
  const hipError_t e = ckda::launch_linattn_bwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

int ckda_linattn_decode_step(const void* q, const void* k, const void* v, const void* g, float* H_inout, void* o, int N,
                             int H, int Hk, int dk, int dv, int dtype, int flags, void* stream) {
  const char* fn = "ckda_linattn_decode_step";
  int st = linattn_sizes(fn, N, H, Hk, 1, dk, dv, dtype, flags);
  if (st != CKDA_OK) return st;
  const size_t NH = (size_t)N * H;
  if (NH == 0) return ok();
  if (NH >= 1u << 24) return fail(CKDA_ERR_DIM, "%s: N*H exceeds the launch grid", fn);   // 256 threads each, of 2^32
  if (!q || !k || !v || !g || !H_inout || !o) return fail(CKDA_ERR_NULL, "%s: every pointer is required", fn);
  const LinAttnSizes n = linattn_bytes(N, H, Hk, 1, dk, dv, dtype, flags);
  const Range in[] = {range("q", q, n.qk), range("k", k, n.qk), range("v", v, n.v), range("g", g, n.g)};
  const Range out[] = {range("o", o, n.v), range("H_inout", H_inout, n.states)};
  if ((st = check_aligned(fn, in, 4)) != CKDA_OK || (st = check_aligned(fn, out, 2)) != CKDA_OK) return st;
  if ((st = check_alias(fn, in, 4, out, 2, nullptr)) != CKDA_OK) return st;
  const ckda::LinAttnDecodeArgs a{q,  k,  v,     g, H_inout, o, N, H, Hk, dk, dv, dtype, (flags & CKDA_DECAY_HEAD) != 0,
                                  (hipStream_t)stream};
  const hipError_t e = ckda::launch_linattn_decode(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

// ---------------------------------------------------------------- head norm

constexpr int kNormMaxD = 8192;
constexpr int kNormActs = CKDA_NORM_GATE_SILU | CKDA_NORM_GATE_SIGMOID;

static int head_norm_sizes(const char* fn, const void* z, int B, int H, int T, int D, int wheads, int dtype, int flags,
                           float eps) {
  if ((flags & ~(CKDA_NORM_RMS | kNormActs)) != 0)
    return fail(CKDA_ERR_FLAGS, "%s: flags 0x%x has bits outside CKDA_NORM_* (0x%x)", fn, flags,
                CKDA_NORM_RMS | kNormActs);
  if (B < 0 || H < 0 || T < 0 || D < 1)
    return fail(CKDA_ERR_DIM, "%s: negative or empty size (B=%d H=%d T=%d D=%d)", fn, B, H, T, D);
  const int acts = flags & kNormActs;
  if (acts == kNormActs || (acts && !z) || (z && !acts))
    return fail(CKDA_ERR_FLAGS, "%s: a gate z takes exactly one of CKDA_NORM_GATE_SILU and _SIGMOID (flags 0x%x, z %s)",
                fn, flags, z ? "given" : "NULL");
  if (wheads != 1 && wheads != H) return fail(CKDA_ERR_DIM, "%s: wheads=%d is neither 1 nor H=%d", fn, wheads, H);
  if (!supported_dtype(dtype)) return fail(CKDA_ERR_UNSUPPORTED, "%s: dtype %d is not F32(0) or BF16(1)", fn, dtype);
  if (D > kNormMaxD) return fail(CKDA_ERR_UNSUPPORTED, "%s: D=%d (supported: 1 .. %d)", fn, D, kNormMaxD);
  if (!(eps > 0.f) || eps > 3.4e38f) return fail(CKDA_ERR_DIM, "%s: eps=%g is not finite and positive", fn, (double)eps);
  if ((size_t)B * T > (size_t)INT32_MAX / 2 || H > 65535)
    return fail(CKDA_ERR_DIM, "%s: B*T or H exceeds the launch grid", fn);
  return CKDA_OK;
}

int ckda_head_norm_fwd(const void* x, const void* z, const float* w, const float* b, void* y, int B, int H, int T,
                       int D, int wheads, int dtype, int flags, float eps, void* stream) {
  const char* fn = "ckda_head_norm_fwd";
  int st = head_norm_sizes(fn, z, B, H, T, D, wheads, dtype, flags, eps);
  if (st != CKDA_OK) return st;
  const size_t rows = (size_t)B * T * H;
  if (rows == 0) return ok();
  if (!x || !y) return fail(CKDA_ERR_NULL, "%s: x and y are required", fn);
  const size_t bytes = rows * D * dtype_bytes(dtype), wb = (size_t)wheads * D * 4;
  const Range in[] = {range("x", x, bytes), range("z", z, z ? bytes : 0), range("w", w, w ? wb : 0),
                      range("b", b, b ? wb : 0)};
  const Range out[] = {range("y", y, bytes)};
  if ((st = check_aligned(fn, in, 4)) != CKDA_OK || (st = check_aligned(fn, out, 1)) != CKDA_OK) return st;
  if ((st = check_alias(fn, in, 4, out, 1, nullptr)) != CKDA_OK) return st;
  ckda::HeadNormArgs a = {};
  a.x = x, a.z = z, a.w = w, a.b = b, a.y = y;
  a.B = B, a.H = H, a.T = T, a.D = D, a.wheads = wheads, a.dtype = dtype, a.flags = flags, a.eps = eps;
  a.stream = (hipStream_t)stream;
  const hipError_t e = ckda::launch_head_norm_fwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

size_t ckda_head_norm_bwd_workspace_size(int B, int H, int T, int D, int wheads, int dtype) {
  if (B < 0 || H < 0 || T < 0 || D < 1 || D > kNormMaxD || (wheads != 1 && wheads != H) || !supported_dtype(dtype))
    return 0;
  if ((size_t)B * T > (size_t)INT32_MAX / 2 || H > 65535) return 0;
  const size_t bytes = ckda::head_norm_bwd_workspace_bytes(B, H, T, D, wheads, dtype);
  return bytes == 0 ? 256 : bytes;
}

int ckda_head_norm_bwd(const void* x, const void* z, const float* w, const float* b, const void* dy, void* dx, void* dz,
                       float* dw, float* db, int B, int H, int T, int D, int wheads, int dtype, int flags, float eps,
                       void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "ckda_head_norm_bwd";
  int st = head_norm_sizes(fn, z, B, H, T, D, wheads, dtype, flags, eps);
  if (st != CKDA_OK) return st;
  const size_t rows = (size_t)B * T * H;
  // gradients of shared weights exist (as zeros) without rows or heads
  if (wheads == 0 || (rows == 0 && !dw && !db)) return ok();
  if (rows > 0 && (!x || !dy || !dx || (z && !dz)))
    return fail(CKDA_ERR_NULL, "%s: x, dy and dx (dz with z) are required", fn);
  const size_t need = ckda_head_norm_bwd_workspace_size(B, H, T, D, wheads, dtype);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const size_t bytes = rows * D * dtype_bytes(dtype), wb = (size_t)wheads * D * 4;
  const Range in[] = {range("x", x, bytes), range("z", z, z ? bytes : 0), range("w", w, w ? wb : 0),
                      range("b", b, b ? wb : 0), range("dy", dy, bytes), range("workspace", workspace, need)};
  const Range out[] = {range("dx", dx, bytes), range("dz", dz, z ? bytes : 0), range("dw", dw, dw ? wb : 0),
                       range("db", db, db ? wb : 0)};
  if ((st = check_aligned(fn, in, 6)) != CKDA_OK || (st = check_aligned(fn, out, 4)) != CKDA_OK) return st;
  if ((st = check_alias(fn, in, 6, out, 4, &in[5])) != CKDA_OK) return st;
  ckda::HeadNormArgs a = {};
  a.x = x, a.z = z, a.w = w, a.b = b, a.dy = dy, a.dx = dx, a.dz = dz, a.dw = dw, a.db = db;
  a.B = B, a.H = H, a.T = T, a.D = D, a.wheads = wheads, a.dtype = dtype, a.flags = flags, a.eps = eps;
  a.workspace = workspace, a.stream = (hipStream_t)stream;
  const hipError_t e = ckda::launch_head_norm_bwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

}  // extern "C"
