// kd_pad.hpp -- zero-padded copies of matrix operands.
#pragma once

#include "kd_gemm.hpp"

namespace kd {

// dst[r][c] = src[r][c] for r < rows, c < cols; zero elsewhere in the
// [dst_rows x ld_dst] destination.
template <class E>
__global__ __launch_bounds__(256) void pad_kernel(const typename E::T* src, int64_t ld_src, int64_t rows,
                                                  int64_t cols, typename E::T* dst, int64_t ld_dst,
                                                  int64_t dst_rows) {
  typedef typename E::T T;
  const int64_t n = dst_rows * ld_dst;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / ld_dst, c = i - r * ld_dst;
    dst[i] = (r < rows && c < cols) ? src[r * ld_src + c] : (T)0;
  }
}

}  // namespace kd
