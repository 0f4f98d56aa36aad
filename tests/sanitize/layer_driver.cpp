// Drives the entry points of the short convolution, the selective scan and the norm
// with the residual's addition through their argument checks, their splits of the
// work over many sizes and, when no GPU is visible, on through the host side of their
// launches (which then fail with CKDA_ERR_HIP), for a build of the host code with
// AddressSanitizer and UndefinedBehaviorSanitizer (tests/test_layer_host_sanitizer.py).
// Device pointers are fake addresses that the host code never dereferences.  Exit
// status 0 means every call returned the expected status.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "ckda.h"

static int failures = 0;
static void expect(long long got, long long want, const char* what, int line) {
  if (got != want) {
    fprintf(stderr, "line %d: %s returned %lld, expected %lld (%s)\n", line, what, got, want, ckda_last_error());
    ++failures;
  }
}
#define EXPECT(call, want) expect((long long)(call), (want), #call, __LINE__)

static void* P(uintptr_t gb) { return (void*)((uintptr_t)0x7F0000000000ull + (gb << 42)); }   // 4 TiB apart
static float* F(uintptr_t gb) { return (float*)P(gb); }
static bool done_or_refused(int st) { return st == CKDA_ERR_HIP || st == CKDA_ERR_DIM || st == CKDA_ERR_ALIAS; }

int main() {
  int ndev = 0;
  const bool gpu = hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0;
  const size_t huge = (size_t)1 << 41;
  const int batches[] = {0, 1, 3, 64, 1000, 70000, 1 << 24, INT_MAX};
  const int lengths[] = {0, 1, 15, 16, 17, 129, 4096, 32768, 1 << 20, 1 << 26, INT_MAX - 64, INT_MAX};
  const int channels[] = {0, 1, 2, 15, 64, 65, 1000, 2048, 8192, 65537, 1 << 20, (1 << 24) - 1, 1 << 24, INT_MAX};
  for (int B : batches)
    for (int T : lengths)
      for (int C : channels)
        for (int dt = 0; dt < 2; ++dt) {
          for (int K = 1; K <= 5; ++K) {
            const size_t need = ckda_short_conv_bwd_workspace_size(B, T, C, K, dt);
            if (K < 2 || K > 4) EXPECT(need, 0);
            if (gpu || K != 4) continue;
            const int ld = C < INT_MAX - 8 ? C + 8 : C;
            EXPECT(done_or_refused(ckda_short_conv_fwd(P(0), F(1), F(2), P(3), nullptr, P(4), P(5), B, T, C, 1, K, ld, dt, CKDA_CONV_SILU, nullptr)) ||
                   B == 0 || C == 0, 1);
            const int st = ckda_short_conv_bwd(P(0), F(1), F(2), P(3), nullptr, P(4), P(5), P(6), F(7), F(8), P(9), B, T, C, 1, K, ld, dt,
                                               CKDA_PAD_ZERO, P(10), huge, nullptr);
            EXPECT(done_or_refused(st) || st == CKDA_ERR_WORKSPACE || C == 0, 1);
          }
          for (int N : {1, 5, 16, 17, 64, 65})
            for (int G : {1, 2}) {
              const size_t fwd = ckda_selective_scan_fwd_workspace_size(B, T, C, G, N, dt);
              const size_t bwd = ckda_selective_scan_bwd_workspace_size(B, T, C, G, N, dt);
              if (N > 64 || (C % G) != 0) EXPECT(fwd + bwd, 0);
              EXPECT(fwd == 0, bwd == 0);
              if (gpu || C % G != 0 || N > 64) continue;
              int st = ckda_selective_scan_fwd(P(0), P(1), F(2), P(3), P(4), F(5), P(6), F(7), F(8), nullptr, P(9), F(10), B, T, C, G, N, G * N,
                                               C, dt, CKDA_SCAN_SOFTPLUS, P(11), huge, nullptr);
              EXPECT(done_or_refused(st) || st == CKDA_ERR_WORKSPACE || B == 0 || C == 0, 1);
              st = ckda_selective_scan_bwd(P(0), P(1), F(2), P(3), P(4), F(5), P(6), F(7), F(8), nullptr, P(9), F(10), P(11), P(12), F(13), P(14),
                                           P(15), F(16), P(17), F(18), F(19), B, T, C, G, N, G * N, C, dt, 0, P(20), huge, nullptr);
              EXPECT(done_or_refused(st) || st == CKDA_ERR_WORKSPACE || C == 0, 1);
            }
          if (T != 1 || gpu) continue;
          EXPECT(done_or_refused(ckda_short_conv_decode_step(P(0), F(1), F(2), P(3), P(4), B, C, 3, C, dt, 0, nullptr)) || B == 0 || C == 0, 1);
          for (int N : {1, 5, 16, 64})
            EXPECT(done_or_refused(ckda_selective_scan_decode_step(P(0), P(1), F(2), P(3), P(4), F(5), P(6), F(7), F(8), P(9), B, C, 1, N, N, C, dt,
                                                                   0, nullptr)) || B == 0 || C == 0, 1);
        }
  EXPECT(ckda_selective_scan_fwd(P(0), P(1), F(2), P(3), P(4), nullptr, nullptr, nullptr, nullptr, nullptr, P(9), nullptr, 1, 1, 64, INT_MAX, 64,
                                 64, 64, 1, 0, P(11), huge, nullptr), CKDA_ERR_DIM);
  EXPECT(ckda_selective_scan_fwd(P(0), P(1), F(2), P(3), P(4), nullptr, nullptr, nullptr, nullptr, nullptr, P(9), nullptr, 1, 1, 0, INT_MAX, 64,
                                 INT_MAX, 0, 1, 0, P(11), huge, nullptr), CKDA_ERR_DIM);
  for (int D : {1, 7, 8, 64, 129, 512, 513, 1024, 1025, 2049, 4097, 8191, 8192, 8193})
    for (int R : {0, 1, 5, 1000, 70000, 1 << 24, INT_MAX})
      for (int dt = 0; dt < 2; ++dt)
        for (int rt = 0; rt < 2; ++rt) {
          const bool good = D <= 8192 && (rt == 0 || rt == dt);
          EXPECT(ckda_add_norm_bwd_workspace_size(R, D, dt, rt) > 0, good);
          if (gpu || R == INT_MAX) continue;   // (the tensors would reach into each other)
          for (int group : {0, 128}) {
            const int st = ckda_add_norm_fwd(P(0), P(1), F(2), P(3), P(4), F(5), P(6), R, D, group, dt, rt, 1e-6f, nullptr);
            EXPECT(st, !good ? CKDA_ERR_UNSUPPORTED : R == 0 ? CKDA_OK : CKDA_ERR_HIP);
          }
          const int st = ckda_add_norm_bwd(P(0), F(1), P(2), P(3), P(4), P(5), F(6), R, D, dt, rt, 1e-6f, P(7), huge, nullptr);
          EXPECT(st, good ? CKDA_ERR_HIP : CKDA_ERR_UNSUPPORTED);
        }
  printf("layer driver (%s): %d failures\n", gpu ? "GPU visible: argument checks only" : "no GPU", failures);
  return failures ? 1 : 0;
}
