// kd_order.hpp -- ordering of logits: order-preserving integer keys and an
// in-LDS sort, shared by the cache builder and sampling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kd {

// Order-preserving unsigned keys of fp32 values (larger float, larger key).
__device__ __forceinline__ uint32_t fkey(float f) {
  const uint32_t b = __float_as_uint(f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float fkey_inv(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// Sort key of a candidate: z descending, then id ascending, as one uint64
// (larger = earlier).
__device__ __forceinline__ uint64_t cand_key(float z, uint32_t id) {
  return ((uint64_t)fkey(z) << 32) | (uint64_t)(0xffffffffu - id);
}

// In-LDS bitonic sort of n (a power of two) uint64 keys, descending.
__device__ __forceinline__ void bitonic_desc(uint64_t* s, int n) {
  for (int size = 2; size <= n; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = threadIdx.x; i < (n >> 1); i += blockDim.x) {
        const int lo = 2 * i - (i & (stride - 1));
        const int hi = lo + stride;
        const bool desc = ((lo & size) == 0);
        const uint64_t a = s[lo], b = s[hi];
        if ((a < b) == desc) {
          s[lo] = b;
          s[hi] = a;
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace kd
