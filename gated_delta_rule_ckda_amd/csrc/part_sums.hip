// part_sums.hip -- column sums of the fp32 parts that workgroups leave behind
// (gradients of weights), in a fixed order.
//
// One workgroup sums 16 columns: 64 threads on each take every 64th part, and
// join through LDS by halves.  16 columns are one 64-byte piece of each part; a
// thread has four parts' loads in flight.  Latency-bound at the sizes that occur
// (a few MB from the last-level cache).
#include "ckda_internal.hpp"

namespace ckda {

namespace {

constexpr int kCols = 16, kRows = 64;

struct Outs {
  float* out[3];
  size_t end[3];   // columns up to and with output i
};

__global__ __launch_bounds__(kCols * kRows) void part_sums_kernel(const float* part, int nparts, size_t stride, Outs o) {
  __shared__ float s[kRows][kCols + 1];
  const int tid = threadIdx.x, j = tid / kCols;
  const size_t c = (size_t)blockIdx.x * kCols + tid % kCols;
  float x = 0.f;
  if (c < o.end[2]) {
#pragma unroll 4
    for (int i = j; i < nparts; i += kRows) x += part[(size_t)i * stride + c];
  }
  s[j][tid % kCols] = x;
  __syncthreads();
  for (int half = kRows / 2; half > 0; half >>= 1) {
    if (j < half) s[j][tid % kCols] += s[j + half][tid % kCols];
    __syncthreads();
  }
  if (j != 0 || c >= o.end[2]) return;
  const int which = c < o.end[0] ? 0 : c < o.end[1] ? 1 : 2;
  float* out = o.out[which];
  if (out) out[c - (which ? o.end[which - 1] : 0)] = s[0][tid];
}

}  // namespace

hipError_t launch_part_sums(const PartSums& p, hipStream_t stream) {
  Outs o;
  size_t end = 0;
  for (int i = 0; i < 3; ++i) {
    o.out[i] = p.out[i];
    o.end[i] = end += p.cols[i];
  }
  if (end == 0 || (!p.out[0] && !p.out[1] && !p.out[2])) return hipSuccess;
  hipLaunchKernelGGL(part_sums_kernel, dim3((unsigned)((end + kCols - 1) / kCols)), dim3(kCols * kRows), 0, stream, p.part,
                     p.nparts, p.stride, o);
  return hipGetLastError();
}

}  // namespace ckda
