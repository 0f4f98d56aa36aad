// part_sums.hip -- the sums of part_sums.hpp as a launch of their own.
#include "part_sums.hpp"

namespace ckda {

namespace {

constexpr int kSumRows = 64;

__global__ __launch_bounds__(kSumCols * kSumRows) void part_sums_kernel(SumOuts o) { sum_parts<kSumRows>(o, blockIdx.x); }

}  // namespace

hipError_t launch_part_sums(const PartSums& p, hipStream_t stream) {
  const SumOuts o = sum_outs(p);
  if (!wanted(o)) return hipSuccess;
  hipLaunchKernelGGL(part_sums_kernel, dim3(sum_blocks(o)), dim3(kSumCols * kSumRows), 0, stream, o);
  return hipGetLastError();
}

}  // namespace ckda
