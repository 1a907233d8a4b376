// kd_rows.hpp -- row access shared by the streaming operators (layer norm,
// 8-bit checkpoints, head logits of few rows, sampling): eight consecutive
// elements of a row per lane, wherever the row starts.
//
// Rows may start at any multiple of the element size (a width that is odd
// puts every second bf16 row at an address that is 2 mod 4): the 16-byte
// loads and stores are written as copies of element alignment, for which
// gfx950 still issues one 128-bit access.  A vector that crosses the end of
// its row is read and written element by element, so nothing outside the row
// is touched.
#pragma once

#include "kd_gemm.hpp"

namespace kd {

struct Vec8 { float v[8]; };

__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
  u32x4 u;
  __builtin_memcpy(&u, p, 16);
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(u[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ Vec8 load8(const float* p) {
  f32x4 a, b;
  __builtin_memcpy(&a, p, 16);
  __builtin_memcpy(&b, p + 4, 16);
  return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ Vec8 load8(const int8_t* p) {
  uint32_t u[2];
  __builtin_memcpy(u, p, 8);
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = (float)(int8_t)(u[i >> 2] >> (8 * (i & 3)));
  return r;
}
__device__ __forceinline__ void store8(uint16_t* p, const Vec8& x) {
  const u32x4 u = {pack_bf16x2(x.v[0], x.v[1]), pack_bf16x2(x.v[2], x.v[3]), pack_bf16x2(x.v[4], x.v[5]),
                   pack_bf16x2(x.v[6], x.v[7])};
  __builtin_memcpy(p, &u, 16);
}
__device__ __forceinline__ void store8(float* p, const Vec8& x) {
  const f32x4 a = {x.v[0], x.v[1], x.v[2], x.v[3]}, b = {x.v[4], x.v[5], x.v[6], x.v[7]};
  __builtin_memcpy(p, &a, 16);
  __builtin_memcpy(p + 4, &b, 16);
}

__device__ __forceinline__ float widen(uint16_t b) { return bf16_to_f32(b); }
__device__ __forceinline__ float widen(float f) { return f; }
__device__ __forceinline__ float widen(int8_t q) { return (float)q; }
__device__ __forceinline__ void narrow(uint16_t* p, float f) { *p = f32_to_bf16(f); }
__device__ __forceinline__ void narrow(float* p, float f) { *p = f; }

// Elements c .. c + 7 of a row of d (zeros past its end).
template <class T>
__device__ __forceinline__ Vec8 row_load8(const T* row, int c, int d) {
  if (c + 8 <= d) return load8(row + c);
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = c + i < d ? widen(row[c + i]) : 0.f;
  return r;
}
template <class T>
__device__ __forceinline__ void row_store8(T* row, int c, int d, const Vec8& x) {
  if (c + 8 <= d) {
    store8(row + c, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < d) narrow(row + c + i, x.v[i]);
  }
}

// Sum over the 64 lanes of a wave, left in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

}  // namespace kd
