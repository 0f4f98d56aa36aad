// row_vec.hpp -- pieces of token-major rows in registers: VEC consecutive
// elements (16 or 8 bytes, or one) at any address that is a multiple of the element's
// size (global memory takes wide accesses at 2-byte boundaries), the last piece of
// a row possibly short.  Device code.
#pragma once

#include "ckda_device.hpp"

namespace ckda {

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);   // elements in 16 bytes

// VEC elements as loaded.  `left` is how many of them the row still has (<= 0:
// none, and nothing is read); the others are zero.  Every load and store is a branch
// on the piece being whole, with the elements of a short one beside it.
template <typename T, int VEC> struct RowVec {
  static_assert(VEC * sizeof(T) == 16 || VEC * sizeof(T) == 8 || VEC == 1, "piece of a row");
  T e[VEC];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(0.f);
  }
  __device__ __forceinline__ void load(const T* p, int left) {
    if (left >= VEC) {
      __builtin_memcpy(e, p, sizeof(e));
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = i < left ? p[i] : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void store(T* p, int left) const {
    if (left >= VEC) {
      __builtin_memcpy(p, e, sizeof(e));
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < left) p[i] = e[i];
    }
  }
  __device__ __forceinline__ void widen(float* v) const {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = to_f32(e[i]);
  }
  __device__ __forceinline__ void round(const float* v) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(v[i]);
  }
};

// sigmoid(z).  Where the result is rounded to bf16, by the hardware's exp2 and
// reciprocal (a few 2^-23, against a rounding of 2^-8).
template <typename T> __device__ __forceinline__ float row_sigmoid(float z) {
  if constexpr (sizeof(T) == 2)
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
  else return 1.f / (1.f + expf(-z));
}
// d/du of u sigmoid(u), given sigmoid(u)
__device__ __forceinline__ float silu_slope(float u, float sg) { return sg * __builtin_fmaf(u, 1.f - sg, 1.f); }

}  // namespace ckda
