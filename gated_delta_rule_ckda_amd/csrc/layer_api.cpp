// layer_api.cpp -- the C ABI of what stands around a recurrence in a layer: the
// short causal convolution, the selective scan and the norm with the residual's
// addition (include/ckda.h).  Argument, aliasing and workspace checks, dispatch and
// error reporting; as in ckda_api.cpp nothing here touches device memory and every
// check runs before a launch.
#include "ckda_checks.hpp"
#include "ckda_internal.hpp"

using namespace ckda;

namespace {

constexpr int kMostChannels = 1 << 24;

// bytes from the first element to behind the last of `rows` rows of `width`
// elements, `ld` apart
size_t span(size_t rows, size_t width, size_t ld, size_t es) { return rows ? ((rows - 1) * ld + width) * es : 0; }

int check_element(const char* fn, const char* name, const void* p, size_t es) {
  if (((uintptr_t)p & (es - 1)) != 0) return fail(CKDA_ERR_DIM, "%s: %s is not %zu-byte aligned", fn, name, es);
  return CKDA_OK;
}

int check_eps(const char* fn, float eps) {
  if (!(eps > 0.f) || eps > 3.4e38f) return fail(CKDA_ERR_DIM, "%s: eps=%g is not finite and positive", fn, (double)eps);
  return CKDA_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- short convolution

static int conv_sizes(const char* fn, int B, int T, int C, int H, int K, int ldx, int dtype, int flags, int known) {
  if ((flags & ~known) != 0) return fail(CKDA_ERR_FLAGS, "%s: flags 0x%x has bits outside 0x%x", fn, flags, known);
  if (B < 0 || T < 0 || C < 0) return fail(CKDA_ERR_DIM, "%s: negative size (B=%d T=%d C=%d)", fn, B, T, C);
  if (H < 1 || C % H != 0) return fail(CKDA_ERR_DIM, "%s: H=%d does not divide C=%d", fn, H, C);
  if (ldx < C) return fail(CKDA_ERR_DIM, "%s: row stride ldx=%d below C=%d", fn, ldx, C);
  if (K < 2 || K > 4) return fail(CKDA_ERR_UNSUPPORTED, "%s: K=%d (supported: 2, 3, 4)", fn, K);
  if (!supported_dtype(dtype)) return fail(CKDA_ERR_UNSUPPORTED, "%s: dtype %d is not F32(0) or BF16(1)", fn, dtype);
  if (C > kMostChannels) return fail(CKDA_ERR_DIM, "%s: C=%d above 2^24", fn, C);
  return CKDA_OK;
}

static int conv_grid(const char* fn, int B, int T, int C, int H) {
  if (T > INT32_MAX - 64 || !short_conv_fits_grid(B, T, C, H)) return fail(CKDA_ERR_DIM, "%s: sizes exceed the launch grid", fn);
  return CKDA_OK;
}

int ckda_short_conv_fwd(const void* x, const float* w, const float* b, const void* s0, const int* lens, void* y,
                        void* sT, int B, int T, int C, int H, int K, int ldx, int dtype, int flags, void* stream) {
  const char* fn = "ckda_short_conv_fwd";
  int st = conv_sizes(fn, B, T, C, H, K, ldx, dtype, flags, CKDA_CONV_SILU | CKDA_PAD_ZERO);
  if (st != CKDA_OK) return st;
  if (B == 0 || C == 0 || (T == 0 && !sT)) return ok();
  if ((T > 0 && (!x || !y)) || !w) return fail(CKDA_ERR_NULL, "%s: x, w and y are required", fn);
  if ((st = conv_grid(fn, B, T, C, H)) != CKDA_OK) return st;
  const size_t es = dtype_bytes(dtype), rows = (size_t)B * T, state = (size_t)B * (K - 1) * C * es;
  const Range in[] = {range("w", w, (size_t)C * K * 4), range("b", b, b ? (size_t)C * 4 : 0),
                      range("s0", s0, s0 ? state : 0), range("x", x, span(rows, C, ldx, es)),
                      range("lens", lens, lens ? (size_t)B * 4 : 0)};
  const Range out[] = {range("y", y, rows * C * es), range("sT", sT, sT ? state : 0)};
  if ((st = check_aligned(fn, in, 3)) != CKDA_OK || (st = check_aligned(fn, out, 2)) != CKDA_OK) return st;
  if ((st = check_element(fn, "x", x, es)) != CKDA_OK || (st = check_element(fn, "lens", lens, 4)) != CKDA_OK) return st;
  if ((st = check_alias(fn, in, 5, out, 2, nullptr)) != CKDA_OK) return st;
  ShortConvArgs a = {};
  a.x = x, a.w = w, a.b = b, a.s0 = s0, a.lens = lens, a.y = y, a.sT = sT;
  a.B = B, a.T = T, a.C = C, a.H = H, a.K = K, a.ldx = ldx, a.dtype = dtype;
  a.silu = (flags & CKDA_CONV_SILU) != 0, a.pad_zero = (flags & CKDA_PAD_ZERO) != 0;
  a.stream = (hipStream_t)stream;
  const hipError_t e = launch_short_conv_fwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

size_t ckda_short_conv_bwd_workspace_size(int B, int T, int C, int K, int dtype) {
  if (B < 0 || T < 0 || C < 0 || K < 2 || K > 4 || !supported_dtype(dtype) || C > kMostChannels) return 0;
  if (T > INT32_MAX - 64 || !short_conv_fits_grid(B, T, C, 1)) return 0;
  const size_t bytes = short_conv_bwd_workspace_bytes(B, T, C, K);
  return bytes < 256 ? 256 : bytes;
}

int ckda_short_conv_bwd(const void* x, const float* w, const float* b, const void* s0, const int* lens, const void* dy,
                        const void* dsT, void* dx, float* dw, float* db, void* ds0, int B, int T, int C, int H, int K,
                        int ldx, int dtype, int flags, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "ckda_short_conv_bwd";
  int st = conv_sizes(fn, B, T, C, H, K, ldx, dtype, flags, CKDA_CONV_SILU | CKDA_PAD_ZERO);
  if (st != CKDA_OK) return st;
  if (C == 0 || ((B == 0 || T == 0) && !dw && !db && (B == 0 || !ds0))) return ok();
  if ((B > 0 && T > 0 && (!x || !dy || !dx)) || !w) return fail(CKDA_ERR_NULL, "%s: x, w, dy and dx are required", fn);
  if ((st = conv_grid(fn, B, T, C, H)) != CKDA_OK) return st;
  const size_t need = ckda_short_conv_bwd_workspace_size(B, T, C, K, dtype);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const size_t es = dtype_bytes(dtype), rows = (size_t)B * T, state = (size_t)B * (K - 1) * C * es;
  const size_t wb = (size_t)C * K * 4, bb = (size_t)C * 4;
  const Range in[] = {range("w", w, wb), range("b", b, b ? bb : 0), range("s0", s0, s0 ? state : 0),
                      range("dy", dy, rows * C * es), range("dsT", dsT, dsT ? state : 0),
                      range("workspace", workspace, need), range("x", x, span(rows, C, ldx, es)),
                      range("lens", lens, lens ? (size_t)B * 4 : 0)};
  const Range out[] = {range("dx", dx, rows * C * es), range("dw", dw, dw ? wb : 0), range("db", db, db ? bb : 0),
                       range("ds0", ds0, ds0 ? state : 0)};
  if ((st = check_aligned(fn, in, 6)) != CKDA_OK || (st = check_aligned(fn, out, 4)) != CKDA_OK) return st;
  if ((st = check_element(fn, "x", x, es)) != CKDA_OK || (st = check_element(fn, "lens", lens, 4)) != CKDA_OK) return st;
  if ((st = check_alias(fn, in, 8, out, 4, &in[5])) != CKDA_OK) return st;
  ShortConvArgs a = {};
  a.x = x, a.w = w, a.b = b, a.s0 = s0, a.lens = lens, a.dy = dy, a.dsT = dsT, a.dx = dx, a.dw = dw, a.db = db, a.ds0 = ds0;
  a.B = B, a.T = T, a.C = C, a.H = H, a.K = K, a.ldx = ldx, a.dtype = dtype;
  a.silu = (flags & CKDA_CONV_SILU) != 0, a.pad_zero = (flags & CKDA_PAD_ZERO) != 0;
  a.workspace = workspace, a.stream = (hipStream_t)stream;
  const hipError_t e = launch_short_conv_bwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

int ckda_short_conv_decode_step(const void* x, const float* w, const float* b, void* state_inout, void* y, int N, int C,
                                int K, int ldx, int dtype, int flags, void* stream) {
  const char* fn = "ckda_short_conv_decode_step";
  int st = conv_sizes(fn, N, 1, C, 1, K, ldx, dtype, flags, CKDA_CONV_SILU);
  if (st != CKDA_OK) return st;
  if (N == 0 || C == 0) return ok();
  if (!x || !w || !state_inout || !y) return fail(CKDA_ERR_NULL, "%s: x, w, state_inout and y are required", fn);
  if ((size_t)N * C >= (size_t)1 << 31) return fail(CKDA_ERR_DIM, "%s: N*C exceeds the launch grid", fn);
  const size_t es = dtype_bytes(dtype);
  const Range in[] = {range("w", w, (size_t)C * K * 4), range("b", b, b ? (size_t)C * 4 : 0),
                      range("x", x, span(N, C, ldx, es))};
  const Range out[] = {range("state_inout", state_inout, (size_t)N * (K - 1) * C * es), range("y", y, (size_t)N * C * es)};
  if ((st = check_aligned(fn, in, 2)) != CKDA_OK || (st = check_aligned(fn, out, 2)) != CKDA_OK) return st;
  if ((st = check_element(fn, "x", x, es)) != CKDA_OK) return st;
  if ((st = check_alias(fn, in, 3, out, 2, nullptr)) != CKDA_OK) return st;
  ShortConvArgs a = {};
  a.x = x, a.w = w, a.b = b, a.y = y, a.state = state_inout;
  a.B = N, a.T = 1, a.C = C, a.H = 1, a.K = K, a.ldx = ldx, a.dtype = dtype;
  a.silu = (flags & CKDA_CONV_SILU) != 0, a.stream = (hipStream_t)stream;
  const hipError_t e = launch_short_conv_decode(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

// ---------------------------------------------------------------- selective scan

static int scan_check(const char* fn, int B, int T, int C, int G, int N, int ldbc, int ldz, bool gate, int dtype, int flags,
                      int known) {
  if ((flags & ~known) != 0) return fail(CKDA_ERR_FLAGS, "%s: flags 0x%x has bits outside 0x%x", fn, flags, known);
  if (B < 0 || T < 0 || C < 0) return fail(CKDA_ERR_DIM, "%s: negative size (B=%d T=%d C=%d)", fn, B, T, C);
  if (G < 1 || C % G != 0) return fail(CKDA_ERR_DIM, "%s: G=%d does not divide C=%d", fn, G, C);
  if (N < 1 || N > 64) return fail(CKDA_ERR_UNSUPPORTED, "%s: N=%d (supported: 1 .. 64)", fn, N);
  if (!supported_dtype(dtype)) return fail(CKDA_ERR_UNSUPPORTED, "%s: dtype %d is not F32(0) or BF16(1)", fn, dtype);
  if (C >= kMostChannels) return fail(CKDA_ERR_DIM, "%s: C=%d not below 2^24", fn, C);
  if ((long long)ldbc < (long long)G * N) return fail(CKDA_ERR_DIM, "%s: row stride ldbc=%d below G*N=%lld", fn, ldbc, (long long)G * N);
  if (gate && ldz < C) return fail(CKDA_ERR_DIM, "%s: row stride ldz=%d below C=%d", fn, ldz, C);
  return CKDA_OK;
}

// the forward's and the backward's tiles of rows take 31-bit offsets; a step's rows, any int
static int scan_strides(const char* fn, int ldbc, int ldz, bool gate) {
  if (ldbc >= kMostChannels || (gate && ldz >= kMostChannels))
    return fail(CKDA_ERR_DIM, "%s: row strides ldbc=%d, ldz=%d must be below 2^24", fn, ldbc, ldz);
  return CKDA_OK;
}

// sizes whose products the host's arithmetic holds and whose launches fit
static bool scan_planned(int B, int T, int C, int G, int N) {
  if (T > INT32_MAX - 64 || (long long)B * C >= 1LL << 31 || (long long)C * N >= 1LL << 28) return false;
  return scan_fits_grid(B, T, C, G, N);
}
static int scan_grid(const char* fn, int B, int T, int C, int G, int N) {
  if (!scan_planned(B, T, C, G, N)) return fail(CKDA_ERR_DIM, "%s: sizes exceed the launch grid", fn);
  return CKDA_OK;
}

static bool scan_sizes_ok(int B, int T, int C, int G, int N, int dtype) {
  return B >= 0 && T >= 0 && C >= 0 && G >= 1 && C % G == 0 && N >= 1 && N <= 64 && supported_dtype(dtype) &&
         C < kMostChannels && scan_planned(B, T, C, G, N);
}

size_t ckda_selective_scan_fwd_workspace_size(int B, int T, int C, int G, int N, int dtype) {
  if (!scan_sizes_ok(B, T, C, G, N, dtype)) return 0;
  const size_t bytes = scan_fwd_workspace_bytes(B, T, C, G, N);
  return bytes < 256 ? 256 : bytes;
}

size_t ckda_selective_scan_bwd_workspace_size(int B, int T, int C, int G, int N, int dtype) {
  if (!scan_sizes_ok(B, T, C, G, N, dtype)) return 0;
  const size_t bytes = scan_bwd_workspace_bytes(B, T, C, G, N);
  return bytes < 256 ? 256 : bytes;
}

int ckda_selective_scan_fwd(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                            const float* D, const void* z, const float* dt_bias, const float* h0, const int* lens,
                            void* y, float* hT, int B, int T, int C, int G, int N, int ldbc, int ldz, int dtype,
                            int flags, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "ckda_selective_scan_fwd";
  int st = scan_check(fn, B, T, C, G, N, ldbc, ldz, z != nullptr, dtype, flags, CKDA_SCAN_SOFTPLUS | CKDA_PAD_ZERO);
  if (st != CKDA_OK || (st = scan_strides(fn, ldbc, ldz, z != nullptr)) != CKDA_OK) return st;
  if (B == 0 || C == 0 || (T == 0 && !hT)) return ok();
  if (!A || (T > 0 && (!x || !dt || !Bm || !Cm || !y)))
    return fail(CKDA_ERR_NULL, "%s: x, dt, A, Bm, Cm and y are required", fn);
  if ((st = scan_grid(fn, B, T, C, G, N)) != CKDA_OK) return st;
  const size_t need = ckda_selective_scan_fwd_workspace_size(B, T, C, G, N, dtype);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const size_t es = dtype_bytes(dtype), rows = (size_t)B * T, each = rows * C * es, state = (size_t)B * C * N * 4;
  const size_t bc = span(rows, (size_t)G * N, ldbc, es), cb = (size_t)C * 4;
  const Range in[] = {range("x", x, each), range("dt", dt, each), range("A", A, cb * N), range("D", D, D ? cb : 0),
                      range("dt_bias", dt_bias, dt_bias ? cb : 0), range("h0", h0, h0 ? state : 0),
                      range("workspace", workspace, need), range("Bm", Bm, bc), range("Cm", Cm, bc),
                      range("z", z, z ? span(rows, C, ldz, es) : 0), range("lens", lens, lens ? (size_t)B * 4 : 0)};
  const Range out[] = {range("y", y, each), range("hT", hT, hT ? state : 0)};
  if ((st = check_aligned(fn, in, 7)) != CKDA_OK || (st = check_aligned(fn, out, 2)) != CKDA_OK) return st;
  if ((st = check_element(fn, "Bm", Bm, es)) != CKDA_OK || (st = check_element(fn, "Cm", Cm, es)) != CKDA_OK ||
      (st = check_element(fn, "z", z, es)) != CKDA_OK || (st = check_element(fn, "lens", lens, 4)) != CKDA_OK)
    return st;
  if ((st = check_alias(fn, in, 11, out, 2, &in[6], &out[1], &in[5])) != CKDA_OK) return st;   // hT may be h0
  SelScanArgs a = {};
  a.x = x, a.dt = dt, a.A = A, a.Bm = Bm, a.Cm = Cm, a.D = D, a.z = z, a.dt_bias = dt_bias, a.h0 = h0, a.lens = lens;
  a.y = y, a.hT = hT, a.B = B, a.T = T, a.C = C, a.G = G, a.N = N, a.ldbc = ldbc, a.ldz = ldz, a.dtype = dtype;
  a.softplus = (flags & CKDA_SCAN_SOFTPLUS) != 0, a.pad_zero = (flags & CKDA_PAD_ZERO) != 0;
  a.workspace = workspace, a.stream = (hipStream_t)stream;
  const hipError_t e = launch_scan_fwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

int ckda_selective_scan_bwd(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                            const float* D, const void* z, const float* dt_bias, const float* h0, const int* lens,
                            const void* dy, const float* dhT, void* dx, void* ddt, float* dA, void* dBm, void* dCm,
                            float* dD, void* dz, float* ddt_bias, float* dh0, int B, int T, int C, int G, int N,
                            int ldbc, int ldz, int dtype, int flags, void* workspace, size_t workspace_bytes,
                            void* stream) {
  const char* fn = "ckda_selective_scan_bwd";
  int st = scan_check(fn, B, T, C, G, N, ldbc, ldz, z != nullptr, dtype, flags, CKDA_SCAN_SOFTPLUS | CKDA_PAD_ZERO);
  if (st != CKDA_OK || (st = scan_strides(fn, ldbc, ldz, z != nullptr)) != CKDA_OK) return st;
  const bool rows_there = B > 0 && T > 0;
  // gradients of the weights exist (as zeros) without rows, and so does the initial state's; dBm and dCm are
  // zero where there are rows but no channels
  if (!rows_there && (C == 0 || (!dA && !dD && !ddt_bias && (B == 0 || !dh0)))) return ok();
  if ((C > 0 && !A) || (rows_there && (!dBm || !dCm)) ||
      (rows_there && C > 0 && (!x || !dt || !Bm || !Cm || !dy || !dx || !ddt || (z && !dz))))
    return fail(CKDA_ERR_NULL, "%s: x, dt, A, Bm, Cm, dy and the gradients of x, dt, Bm, Cm (and z) are required", fn);
  if ((st = scan_grid(fn, B, T, C, G, N)) != CKDA_OK) return st;
  const size_t need = ckda_selective_scan_bwd_workspace_size(B, T, C, G, N, dtype);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const size_t es = dtype_bytes(dtype), rows = (size_t)B * T, each = rows * C * es, state = (size_t)B * C * N * 4;
  const size_t bc = span(rows, (size_t)G * N, ldbc, es), cb = (size_t)C * 4, dbc = rows * G * N * es;
  const Range in[] = {range("x", x, each), range("dt", dt, each), range("A", A, cb * N), range("D", D, D ? cb : 0),
                      range("dt_bias", dt_bias, dt_bias ? cb : 0), range("h0", h0, h0 ? state : 0),
                      range("dy", dy, each), range("dhT", dhT, dhT ? state : 0), range("workspace", workspace, need),
                      range("Bm", Bm, bc), range("Cm", Cm, bc), range("z", z, z ? span(rows, C, ldz, es) : 0),
                      range("lens", lens, lens ? (size_t)B * 4 : 0)};
  const Range out[] = {range("dx", dx, each), range("ddt", ddt, each), range("dA", dA, dA ? cb * N : 0),
                       range("dBm", dBm, dbc), range("dCm", dCm, dbc), range("dD", dD, dD ? cb : 0),
                       range("dz", dz, z ? each : 0), range("ddt_bias", ddt_bias, ddt_bias ? cb : 0),
                       range("dh0", dh0, dh0 ? state : 0)};
  if ((st = check_aligned(fn, in, 9)) != CKDA_OK || (st = check_aligned(fn, out, 9)) != CKDA_OK) return st;
  if ((st = check_element(fn, "Bm", Bm, es)) != CKDA_OK || (st = check_element(fn, "Cm", Cm, es)) != CKDA_OK ||
      (st = check_element(fn, "z", z, es)) != CKDA_OK || (st = check_element(fn, "lens", lens, 4)) != CKDA_OK)
    return st;
  if ((st = check_alias(fn, in, 13, out, 9, &in[8])) != CKDA_OK) return st;
  SelScanArgs a = {};
  a.x = x, a.dt = dt, a.A = A, a.Bm = Bm, a.Cm = Cm, a.D = D, a.z = z, a.dt_bias = dt_bias, a.h0 = h0, a.lens = lens;
  a.dy = dy, a.dhT = dhT, a.dx = dx, a.ddt = ddt, a.dA = dA, a.dBm = dBm, a.dCm = dCm, a.dD = dD, a.dz = dz;
  a.dbias = ddt_bias, a.dh0 = dh0;
  a.B = B, a.T = T, a.C = C, a.G = G, a.N = N, a.ldbc = ldbc, a.ldz = ldz, a.dtype = dtype;
  a.softplus = (flags & CKDA_SCAN_SOFTPLUS) != 0, a.pad_zero = (flags & CKDA_PAD_ZERO) != 0;
  a.workspace = workspace, a.stream = (hipStream_t)stream;
  const hipError_t e = launch_scan_bwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

int ckda_selective_scan_decode_step(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm,
                                    const float* D, const void* z, const float* dt_bias, float* H_inout, void* y, int S,
                                    int C, int G, int N, int ldbc, int ldz, int dtype, int flags, void* stream) {
  const char* fn = "ckda_selective_scan_decode_step";
  int st = scan_check(fn, S, 1, C, G, N, ldbc, ldz, z != nullptr, dtype, flags, CKDA_SCAN_SOFTPLUS);
  if (st != CKDA_OK) return st;
  if (S == 0 || C == 0) return ok();
  if (!x || !dt || !A || !Bm || !Cm || !H_inout || !y)
    return fail(CKDA_ERR_NULL, "%s: x, dt, A, Bm, Cm, H_inout and y are required", fn);
  if ((size_t)S * C >= (size_t)1 << 27) return fail(CKDA_ERR_DIM, "%s: S*C exceeds the launch grid", fn);
  const size_t es = dtype_bytes(dtype), each = (size_t)S * C * es, bc = span(S, (size_t)G * N, ldbc, es), cb = (size_t)C * 4;
  const Range in[] = {range("x", x, each), range("dt", dt, each), range("A", A, cb * N), range("D", D, D ? cb : 0),
                      range("dt_bias", dt_bias, dt_bias ? cb : 0), range("Bm", Bm, bc), range("Cm", Cm, bc),
                      range("z", z, z ? span(S, C, ldz, es) : 0)};
  const Range out[] = {range("H_inout", H_inout, (size_t)S * C * N * 4), range("y", y, each)};
  if ((st = check_aligned(fn, in, 5)) != CKDA_OK || (st = check_aligned(fn, out, 2)) != CKDA_OK) return st;
  if ((st = check_element(fn, "Bm", Bm, es)) != CKDA_OK || (st = check_element(fn, "Cm", Cm, es)) != CKDA_OK ||
      (st = check_element(fn, "z", z, es)) != CKDA_OK)
    return st;
  if ((st = check_alias(fn, in, 8, out, 2, nullptr)) != CKDA_OK) return st;
  SelScanArgs a = {};
  a.x = x, a.dt = dt, a.A = A, a.Bm = Bm, a.Cm = Cm, a.D = D, a.z = z, a.dt_bias = dt_bias, a.H_inout = H_inout, a.y = y;
  a.B = S, a.T = 1, a.C = C, a.G = G, a.N = N, a.ldbc = ldbc, a.ldz = ldz, a.dtype = dtype;
  a.softplus = (flags & CKDA_SCAN_SOFTPLUS) != 0, a.stream = (hipStream_t)stream;
  const hipError_t e = launch_scan_decode(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

// ---------------------------------------------------------------- norm with the residual's addition

constexpr int kAddNormMaxD = 8192;

static int add_norm_sizes(const char* fn, int R, int D, int dtype, int res_dtype, float eps) {
  if (R < 0 || D < 1) return fail(CKDA_ERR_DIM, "%s: negative or empty size (R=%d D=%d)", fn, R, D);
  if (!supported_dtype(dtype)) return fail(CKDA_ERR_UNSUPPORTED, "%s: dtype %d is not F32(0) or BF16(1)", fn, dtype);
  if (res_dtype != dtype && res_dtype != CKDA_DTYPE_F32)
    return fail(CKDA_ERR_UNSUPPORTED, "%s: res_dtype %d is neither dtype=%d nor F32(0)", fn, res_dtype, dtype);
  if (D > kAddNormMaxD) return fail(CKDA_ERR_UNSUPPORTED, "%s: D=%d (supported: 1 .. %d)", fn, D, kAddNormMaxD);
  return check_eps(fn, eps);
}

int ckda_add_norm_fwd(const void* x, const void* res, const float* w, void* y, void* q, float* scales, void* sum, int R,
                      int D, int group, int dtype, int res_dtype, float eps, void* stream) {
  const char* fn = "ckda_add_norm_fwd";
  int st = add_norm_sizes(fn, R, D, dtype, res_dtype, eps);
  if (st != CKDA_OK) return st;
  if (group != 0 && group != 128) return fail(CKDA_ERR_UNSUPPORTED, "%s: group=%d (supported: 128, or 0 for a row)", fn, group);
  if (R == 0) return ok();
  if (!x || (!y && !q) || (q && !scales) || (!q && scales))
    return fail(CKDA_ERR_NULL, "%s: x and at least one of y and q are required, scales with q", fn);
  const size_t n = (size_t)R * D, es = dtype_bytes(dtype), rs = dtype_bytes(res_dtype);
  const size_t groups = group ? (size_t)(D + group - 1) / group : 1;
  const Range in[] = {range("x", x, n * es), range("res", res, res ? n * rs : 0), range("w", w, w ? (size_t)D * 4 : 0)};
  const Range out[] = {range("y", y, y ? n * es : 0), range("q", q, q ? n : 0),
                       range("scales", scales, scales ? R * groups * 4 : 0), range("sum", sum, sum ? n * rs : 0)};
  if ((st = check_aligned(fn, in, 3)) != CKDA_OK || (st = check_aligned(fn, out, 4)) != CKDA_OK) return st;
  if ((st = check_alias(fn, in, 3, out, 4, nullptr, &out[3], &in[1])) != CKDA_OK) return st;   // sum may be res
  AddNormArgs a = {};
  a.x = x, a.res = res, a.w = w, a.y = y, a.q = q, a.scales = scales, a.sum = sum;
  a.R = R, a.D = D, a.group = group, a.dtype = dtype, a.res_dtype = res_dtype, a.eps = eps, a.stream = (hipStream_t)stream;
  const hipError_t e = launch_add_norm_fwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

size_t ckda_add_norm_bwd_workspace_size(int R, int D, int dtype, int res_dtype) {
  if (R < 0 || D < 1 || D > kAddNormMaxD || !supported_dtype(dtype) || (res_dtype != dtype && res_dtype != CKDA_DTYPE_F32))
    return 0;
  const size_t bytes = add_norm_bwd_workspace_bytes(R, D, dtype);
  return bytes < 256 ? 256 : bytes;
}

int ckda_add_norm_bwd(const void* sum, const float* w, const void* dy, const void* dsum, void* dx, void* dres, float* dw,
                      int R, int D, int dtype, int res_dtype, float eps, void* workspace, size_t workspace_bytes,
                      void* stream) {
  const char* fn = "ckda_add_norm_bwd";
  int st = add_norm_sizes(fn, R, D, dtype, res_dtype, eps);
  if (st != CKDA_OK) return st;
  if (R == 0 && !dw) return ok();
  if (R > 0 && (!sum || !dy || (!dx && !dres)))
    return fail(CKDA_ERR_NULL, "%s: sum, dy and at least one of dx and dres are required", fn);
  const size_t need = ckda_add_norm_bwd_workspace_size(R, D, dtype, res_dtype);
  if ((st = check_workspace(fn, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const size_t n = (size_t)R * D, es = dtype_bytes(dtype), rs = dtype_bytes(res_dtype), wb = (size_t)D * 4;
  const Range in[] = {range("sum", sum, n * rs), range("w", w, w ? wb : 0), range("dy", dy, n * es),
                      range("dsum", dsum, dsum ? n * rs : 0), range("workspace", workspace, need)};
  const Range out[] = {range("dx", dx, dx ? n * es : 0), range("dres", dres, dres ? n * rs : 0),
                       range("dw", dw, dw ? wb : 0)};
  if ((st = check_aligned(fn, in, 5)) != CKDA_OK || (st = check_aligned(fn, out, 3)) != CKDA_OK) return st;
  if ((st = check_alias(fn, in, 5, out, 3, &in[4], &out[1], &in[3])) != CKDA_OK) return st;   // dres may be dsum
  AddNormArgs a = {};
  a.sum = const_cast<void*>(sum), a.w = w, a.dy = dy, a.dsum = dsum, a.dx = dx, a.dres = dres, a.dw = dw;
  a.R = R, a.D = D, a.dtype = dtype, a.res_dtype = res_dtype, a.eps = eps;
  a.workspace = workspace, a.stream = (hipStream_t)stream;
  const hipError_t e = launch_add_norm_bwd(a);
  if (e != hipSuccess) return fail(CKDA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

}  // extern "C"
