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
  Vec8 r = {};
  if (c + 8 <= d) {
    r = load8(row + c);
  } else if (c < d) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < d) r.v[i] = widen(row[c + i]);
  }
  return r;
}
template <class T>
__device__ __forceinline__ void row_store8(T* row, int c, int d, const Vec8& x) {
  if (c + 8 <= d) {
    store8(row + c, x);
  } else if (c < d) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < d) narrow(row + c + i, x.v[i]);
  }
}

// Eight elements as they were loaded: what a kernel that holds a row in
// registers keeps (half of bf16's registers, a quarter of int8's).
template <class T> struct Raw8;
template <> struct Raw8<uint16_t> { u32x4 a; };
template <> struct Raw8<float> { f32x4 a, b; };
template <> struct Raw8<int8_t> { uint32_t a, b; };

template <class T>
__device__ __forceinline__ Raw8<T> raw_load8(const T* p) {
  Raw8<T> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
__device__ __forceinline__ Vec8 unpack(const Raw8<uint16_t>& r) {
  Vec8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.v[2 * i] = __uint_as_float(r.a[i] << 16);
    v.v[2 * i + 1] = __uint_as_float(r.a[i] & 0xffff0000u);
  }
  return v;
}
__device__ __forceinline__ Vec8 unpack(const Raw8<float>& r) {
  return Vec8{{r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w}};
}
__device__ __forceinline__ Vec8 unpack(const Raw8<int8_t>& r) {
  Vec8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v.v[i] = (float)(int8_t)((i < 4 ? r.a : r.b) >> (8 * (i & 3)));
  return v;
}
// The registers as the compiler knows them stay what they are: unpacked again
// at each use rather than kept unpacked.
__device__ __forceinline__ void keep(Raw8<uint16_t>& r) { asm volatile("" : "+v"(r.a)); }
__device__ __forceinline__ void keep(Raw8<float>& r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }
__device__ __forceinline__ void keep(Raw8<int8_t>& r) { asm volatile("" : "+v"(r.a), "+v"(r.b)); }

// Values that are computed by here, not where they are used next (the compiler
// would keep their operands instead).
__device__ __forceinline__ void settle(Vec8& x) {
  asm volatile("" : "+v"(x.v[0]), "+v"(x.v[1]), "+v"(x.v[2]), "+v"(x.v[3]), "+v"(x.v[4]), "+v"(x.v[5]), "+v"(x.v[6]),
               "+v"(x.v[7]));
}
__device__ __forceinline__ void settle(float& a, float& b) { asm volatile("" : "+v"(a), "+v"(b)); }

// ---------------------------------------------------------------------------
// Exchanges between the lanes of a wave, as register moves (DPP): a step
// costs one or two VALU instructions and no LDS round trip.
// ---------------------------------------------------------------------------
constexpr int kDppXor1 = 0xB1;          // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;          // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;   // lane i <- 7 - i of its eight
constexpr int kDppMirror = 0x140;       // lane i <- 15 - i of its sixteen

// The value of the lane that CTRL names; lanes that the move does not reach
// (outside ROWS, or shifted in) get zero bits.  (Where it reaches all, stated
// as bound control, the compiler makes it one instruction with its user.)
template <int CTRL, int ROWS = 0xf, class T>
__device__ __forceinline__ T dpp(T v) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "one or two registers");
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, true));
  } else {
    const int2 u = __builtin_bit_cast(int2, v);
    int2 r;
    r.x = __builtin_amdgcn_update_dpp(0, u.x, CTRL, ROWS, 0xf, true);
    r.y = __builtin_amdgcn_update_dpp(0, u.y, CTRL, ROWS, 0xf, true);
    return __builtin_bit_cast(T, r);
  }
}
template <class T>
__device__ __forceinline__ T read_lane(T v, int lane) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  } else {
    int2 u = __builtin_bit_cast(int2, v);
    u.x = __builtin_amdgcn_readlane(u.x, lane);
    u.y = __builtin_amdgcn_readlane(u.y, lane);
    return __builtin_bit_cast(T, u);
  }
}

// Maximum / sum over each 8 or 16 adjacent lanes, left in all of them.
template <int N, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
  static_assert(N == 8 || N == 16, "lanes that share a result");
  v = op(v, dpp<kDppXor1>(v));
  v = op(v, dpp<kDppXor2>(v));
  v = op(v, dpp<kDppHalfMirror>(v));
  if constexpr (N == 16) v = op(v, dpp<kDppMirror>(v));
  return v;
}
// Over the 64 lanes, the same in all of them; a fixed order of operations.
template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, Op op) {
  v = lanes_reduce<16>(v, op);
  return op(op(read_lane(v, 0), read_lane(v, 16)), op(read_lane(v, 32), read_lane(v, 48)));
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  return wave_reduce(v, [](T a, T b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
// Inclusive prefix sum over the 64 lanes.
template <class T>
__device__ __forceinline__ T wave_incl_scan(T v) {
  v += dpp<0x111>(v);                   // row_shr:1, 2, 4, 8: within sixteen lanes
  v += dpp<0x112>(v);
  v += dpp<0x114>(v);
  v += dpp<0x118>(v);
  v += dpp<0x142, 0xa>(v);              // lane 15 of rows 0 and 2 into rows 1 and 3
  v += dpp<0x143, 0xc>(v);              // lane 31 into rows 2 and 3
  return v;
}

}  // namespace kd
