// part_sums.hpp -- column sums of the fp32 parts that workgroups leave behind
// (gradients of weights), in a fixed order.  Device code.
//
// One workgroup sums 16 columns: ROWS threads on each take every ROWS-th part, and
// join through LDS by halves.  16 columns are one 64-byte piece of each part; a
// thread has four parts' loads in flight.  Latency-bound at the sizes that occur
// (a few MB from the last-level cache).
#pragma once

#include "ckda_internal.hpp"

namespace ckda {

constexpr int kSumCols = 16;

struct SumOuts {
  const float* part;
  int nparts;
  size_t stride;
  float* out[3];
  size_t end[3];   // columns up to and with output i
};
inline SumOuts sum_outs(const PartSums& p) {
  SumOuts o{p.part, p.nparts, p.stride, {}, {}};
  size_t end = 0;
  for (int i = 0; i < 3; ++i) {
    o.out[i] = p.out[i];
    o.end[i] = end += p.cols[i];
  }
  return o;
}
inline bool wanted(const SumOuts& o) { return o.end[2] > 0 && (o.out[0] || o.out[1] || o.out[2]); }
inline unsigned sum_blocks(const SumOuts& o) { return (unsigned)((o.end[2] + kSumCols - 1) / kSumCols); }

// workgroup `block` of sum_blocks, with kSumCols ROWS threads
template <int ROWS> __device__ __forceinline__ void sum_parts(const SumOuts& o, unsigned block) {
  __shared__ float s[ROWS][kSumCols + 1];
  const int tid = threadIdx.x, j = tid / kSumCols;
  const size_t c = (size_t)block * kSumCols + tid % kSumCols;
  float x = 0.f;
  if (c < o.end[2]) {
#pragma unroll 4
    for (int i = j; i < o.nparts; i += ROWS) x += o.part[(size_t)i * o.stride + c];
  }
  s[j][tid % kSumCols] = x;
  __syncthreads();
  for (int half = ROWS / 2; half > 0; half >>= 1) {
    if (j < half) s[j][tid % kSumCols] += s[j + half][tid % kSumCols];
    __syncthreads();
  }
  if (j != 0 || c >= o.end[2]) return;
  const int which = c < o.end[0] ? 0 : c < o.end[1] ? 1 : 2;
  float* out = o.out[which];
  if (out) out[c - (which ? o.end[which - 1] : 0)] = s[0][tid];
}

}  // namespace ckda
