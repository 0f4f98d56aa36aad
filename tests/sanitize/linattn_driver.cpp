// Drives the entry points of the linear attention and of the head norm through
// their argument checks, their splits of the work over many sizes and, when no
// GPU is visible, on through the host side of their launches (which then fail
// with CKDA_ERR_HIP), for a build of the host code with AddressSanitizer and
// UndefinedBehaviorSanitizer (tests/test_linattn_host_sanitizer.py).  Device
// pointers are fake addresses that the host code never dereferences.  Exit
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

static void* P(uintptr_t gb) { return (void*)((uintptr_t)0x7F0000000000ull + (gb << 36)); }   // 64 GiB apart
static float* F(uintptr_t gb) { return (float*)P(gb); }

int main() {
  int ndev = 0;
  const bool gpu = hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0;
  const int widths[] = {16, 32, 64, 128};
  const int heads[] = {1, 2, 7, 16, 33, 64, 100, 256, 513, 4096, 65536, 70000, 1 << 20, 1 << 24};
  const int lengths[] = {0, 1, 63, 64, 65, 129, 200, 777, 1024, 4096, 5001, 32768, 200000, 1 << 20, 1 << 22, 1 << 25, INT_MAX};
  const size_t huge = (size_t)1 << 62;
  // every size: a split, a workspace, and a launch or a refusal
  for (int dk : widths)
    for (int dv : widths)
      for (int h : heads)
        for (int T : lengths)
          for (int dt = 0; dt < 2; ++dt) {
            const bool fits = ((size_t)T + 128) * (dk > dv ? dk : dv) * (dt ? 2 : 4) <= (size_t)INT32_MAX && h * 24ull <= INT32_MAX;
            EXPECT(ckda_linattn_fwd_workspace_size(1, h, T, dk, dv, dt) > 0, fits);
            EXPECT(ckda_linattn_fwd_workspace_size(h, 1, T, dk, dv, dt) > 0, fits);
            if (h % 2 == 0) (void)ckda_linattn_bwd_workspace_size(1, h, h / 2, T, dk, dv, dt);
            (void)ckda_linattn_bwd_workspace_size(h, 1, 1, T, dk, dv, dt);
            if (gpu || h > 600) continue;
            const int st = ckda_linattn_fwd(P(0), P(1), P(2), P(3), F(4), nullptr, P(5), F(6), 1, h, h, T, dk, dv, dt, 0, P(7),
                                            huge >> 20, nullptr);
            EXPECT(st == CKDA_ERR_HIP || st == CKDA_ERR_DIM || st == CKDA_ERR_ALIAS, 1);
            const int sb = ckda_linattn_bwd(P(0), P(1), P(2), P(3), F(4), (const int*)P(5), P(6), F(7), P(8), P(9), P(10), P(11),
                                            F(12), 1, h, 1, T, dk, dv, dt, h % 3 ? CKDA_DECAY_HEAD : 0, P(13), huge, nullptr);
            EXPECT(sb == CKDA_ERR_HIP || sb == CKDA_ERR_DIM || sb == CKDA_ERR_ALIAS, 1);
          }
  EXPECT(ckda_linattn_fwd_workspace_size(INT_MAX, INT_MAX, INT_MAX, 128, 128, 1), 0);
  EXPECT(ckda_linattn_bwd_workspace_size(INT_MAX, INT_MAX, INT_MAX, INT_MAX, 128, 128, 1), 0);
  EXPECT(ckda_linattn_fwd_workspace_size(0, 4, 64, 128, 128, 1), 256);
  EXPECT(ckda_linattn_bwd_workspace_size(1, 4, 3, 64, 128, 128, 1), 0);
  EXPECT(ckda_linattn_fwd(P(0), P(1), P(2), P(3), nullptr, nullptr, P(5), nullptr, INT_MAX, INT_MAX, 1, INT_MAX, 64, 64, 1, 0,
                          P(7), huge, nullptr), CKDA_ERR_DIM);
  EXPECT(ckda_linattn_bwd(P(0), P(1), P(2), P(3), nullptr, nullptr, P(6), nullptr, P(8), P(9), P(10), P(11), nullptr, INT_MAX,
                          INT_MAX, 1, INT_MAX, 64, 64, 1, 0, P(13), huge, nullptr), CKDA_ERR_DIM);
  EXPECT(ckda_linattn_decode_step(P(0), P(1), P(2), P(3), F(4), P(5), INT_MAX, INT_MAX, 1, 128, 128, 1, 0, nullptr),
         CKDA_ERR_DIM);
  EXPECT(ckda_linattn_decode_step(P(0), P(1), P(2), P(3), nullptr, P(5), 1, 1, 1, 128, 128, 1, 0, nullptr), CKDA_ERR_NULL);
  EXPECT(ckda_linattn_decode_step(P(0), P(1), P(2), P(3), F(4), P(4), 1, 1, 1, 128, 128, 1, 0, nullptr), CKDA_ERR_ALIAS);
  if (!gpu)
    for (int dk : widths)
      for (int dv : widths)
        for (int n : heads)
          for (int dt = 0; dt < 2; ++dt) {
            const int st = ckda_linattn_decode_step(P(0), P(1), P(2), P(3), F(8), P(5), n, 1, 1, dk, dv, dt, 0, nullptr);
            EXPECT(st == CKDA_ERR_HIP || (n >= 1 << 20 && st != CKDA_OK), 1);
          }
  // head norm
  const int norm_d[] = {1, 2, 3, 8, 31, 63, 64, 65, 128, 255, 513, 1000, 2047, 4097, 8191, 8192};
  for (int D : norm_d)
    for (int rows : {1, 5, 1000, 70000, INT_MAX / 2})
      for (int H : {1, 3, 16, 65535})
        for (int dt = 0; dt < 2; ++dt) {
          EXPECT(ckda_head_norm_bwd_workspace_size(1, H, rows, D, 1, dt) > 0, 1);
          EXPECT(ckda_head_norm_bwd_workspace_size(rows, H, 1, D, H, dt) > 0, 1);
          if (gpu || rows > 1000 || H > 16) continue;
          EXPECT(ckda_head_norm_fwd(P(0), P(1), F(2), F(3), P(4), 1, H, rows, D, H, dt, CKDA_NORM_GATE_SILU, 1e-5f, nullptr),
                 CKDA_ERR_HIP);
          EXPECT(ckda_head_norm_bwd(P(0), nullptr, F(2), F(3), P(4), P(5), nullptr, F(7), F(8), rows, H, 1, D, 1, dt,
                                    CKDA_NORM_RMS, 1e-5f, P(9), (size_t)1 << 34, nullptr), CKDA_ERR_HIP);
        }
  EXPECT(ckda_head_norm_bwd_workspace_size(INT_MAX, 1, INT_MAX, 64, 1, 1), 0);
  EXPECT(ckda_head_norm_bwd_workspace_size(1, 1, 1, 8193, 1, 1), 0);
  EXPECT(ckda_head_norm_fwd(P(0), nullptr, nullptr, nullptr, P(4), INT_MAX, 1, INT_MAX, 64, 1, 1, 0, 1e-5f, nullptr), CKDA_ERR_DIM);
  EXPECT(ckda_head_norm_fwd(P(0), nullptr, nullptr, nullptr, P(0), 1, 1, 1, 64, 1, 1, 0, 1e-5f, nullptr), CKDA_ERR_ALIAS);
  EXPECT(ckda_head_norm_fwd(P(0), nullptr, nullptr, nullptr, P(4), 1, 1, 1, 64, 1, 1, 0, 0.f, nullptr), CKDA_ERR_DIM);
  printf("linear attention driver (%s): %d failures\n", gpu ? "GPU visible: argument checks only" : "no GPU", failures);
  return failures ? 1 : 0;
}
