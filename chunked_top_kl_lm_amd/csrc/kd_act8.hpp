// kd_act8.hpp -- activation checkpoints in 8 bits: what a backward pass reads
// again of an activation x [T, d], kept as one signed byte per element and
// one fp32 scale per row and block of 128 elements (the last block of a row
// may be shorter).
//
//   s = max(amax * fl(1/127), 2^-126)   amax = largest |x| of the block
//   q = clamp(rint(x * fl(1/s)), -127, 127)
//   x' = q * s
//
// so |x - x'| is at most half a step, amax / 254, and a few fp32 roundings.
// The floor of the scale keeps 1/s finite for blocks of zeros and of
// subnormals.  A block that holds an Inf or a NaN gets the scale NaN and
// comes back as NaN throughout: it is not silently made finite.  One fp32
// division per block; every step is a single correctly rounded operation, so
// the bytes are the same wherever they are computed.
//
// Bound by HBM: (e + 1 + 4/128) bytes per element each way, e the element's
// size.  A lane takes eight consecutive elements, sixteen lanes a block, so
// the block's maximum is four lane exchanges and no LDS; a wave takes up to
// four blocks per load, several loads in flight.
#pragma once

#include "kd_layout.hpp"
#include "kd_rows.hpp"

namespace kd {

// Magnitude bits, doubled, of the largest of eight values (the shift drops
// the sign; a NaN's lie above Inf's, Inf's above every finite value's).
__device__ __forceinline__ uint32_t amax_bits(const Vec8& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x.v[i]) << 1);
  return m;
}
// Maximum over the 16 lanes that share a block, left in each of them.
__device__ __forceinline__ uint32_t block_max16(uint32_t m) {
  return lanes_reduce<16>(m, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// The block's scale from its largest magnitude bits (doubled).
__device__ __forceinline__ float act8_scale(uint32_t amax) {
  if (amax >= 0xff000000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(amax >> 1) * (1.0f / 127.0f), 1.17549435e-38f);
}

// Eight quantised elements as 8 bytes; inv = 1 / scale (NaN: all zero).
// rint by adding 1.5 * 2^23: the sum's low byte is the integer in two's
// complement.  |x * inv| <= 127 (1 + 4 * 2^-24), so the integer needs no
// clamp.  v_perm gathers the bytes, three per four elements.
__device__ __forceinline__ uint2 act8_pack(const Vec8& x, float inv) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float t = x.v[i] * inv;
    asm("" : "+v"(t));                              // two roundings: no fma of product and sum
    b[i] = __float_as_uint(t + 12582912.0f);
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x0c0c0400u);
    w[h] = inv == inv ? lo | (hi << 16) : 0;
  }
  return make_uint2(w[0], w[1]);
}

// One element as a byte.
__device__ __forceinline__ int8_t act8_one(float x, float inv) {
  float t = x * inv;
  asm("" : "+v"(t));
  return inv == inv ? (int8_t)(__float_as_uint(t + 12582912.0f) & 255u) : (int8_t)0;
}

// Quantise the lane's eight elements (c a multiple of 8, the 16 lanes of a
// block adjacent and all active) and write the bytes and, from the block's
// first lane, its scale.  Lanes past the row's end hold zeros and write nothing.
__device__ __forceinline__ void act8_store(const Vec8& x, int8_t* qrow, float* srow, int c, int d) {
  const float s = act8_scale(block_max16(amax_bits(x)));
  const uint2 w = act8_pack(x, 1.0f / s);
  if (c + 8 <= d) {
    __builtin_memcpy(qrow + c, &w, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < d) qrow[c + i] = (int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
  if ((c & (kActBlock - 1)) == 0 && c < d) srow[c / kActBlock] = s;
}

constexpr int kActRows = 4;       // rows (waves) of a block of threads
constexpr int kActSpan = 512;     // elements of a row that a wave takes per load
constexpr int kActLoads = 4;      // loads in flight

// Grid: x = groups of kActRows rows, y = spans of `per` * kActSpan elements
// of each row.
template <class T>
__global__ __launch_bounds__(64 * kActRows) void act8_quantize_kernel(const T* x, int64_t ldx, int64_t rows, int d,
                                                                      int per, int8_t* q, float* scale, int nb) {
  const int64_t t = (int64_t)blockIdx.x * kActRows + (threadIdx.x >> 6);
  if (t >= rows) return;                            // whole waves
  const T* xr = x + t * ldx;
  int8_t* qr = q + t * d;
  float* sr = scale + t * nb;
  const int c0 = blockIdx.y * per * kActSpan, c1 = min(d, c0 + per * kActSpan);
  for (int c = c0; c < c1; c += kActLoads * kActSpan) {
    Vec8 v[kActLoads];
    const int cl = c + 8 * (int)(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < kActLoads; ++i) v[i] = row_load8(xr, cl + i * kActSpan, c1);
#pragma unroll
    for (int i = 0; i < kActLoads; ++i)
      if (c + i * kActSpan < c1) act8_store(v[i], qr, sr, cl + i * kActSpan, c1);
  }
}

// Back to x' (rounded to the output's type).  Rows of ldo elements; with
// rows_pad > rows or ldo > d the padding is written with zeros (what the
// matrix products read).
template <class T>
__global__ __launch_bounds__(64 * kActRows) void act8_dequantize_kernel(const int8_t* q, const float* scale, int nb,
                                                                        int64_t rows, int d, int per, T* out,
                                                                        int64_t ldo, int64_t rows_pad) {
  const int64_t t = (int64_t)blockIdx.x * kActRows + (threadIdx.x >> 6);
  if (t >= rows_pad) return;
  const bool live = t < rows;
  const int8_t* qr = q + (live ? t : 0) * d;
  const float* sr = scale + (live ? t : 0) * nb;
  T* o = out + t * ldo;
  const int c0 = blockIdx.y * per * kActSpan, c1 = min((int)ldo, c0 + per * kActSpan);
  for (int c = c0; c < c1; c += kActLoads * kActSpan) {
    Vec8 v[kActLoads];
    float s[kActLoads];
    const int cl = c + 8 * (int)(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < kActLoads; ++i) {
      const int ci = cl + i * kActSpan;
      v[i] = row_load8(qr, ci, live ? min(d, c1) : 0);
      s[i] = live && ci < d ? sr[ci / kActBlock] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kActLoads; ++i) {
      const int ci = cl + i * kActSpan;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i].v[e] = ci + e < d ? v[i].v[e] * s[i] : 0.f;
      row_store8(o, ci, c1, v[i]);
    }
  }
}

// Spans of a row that the grid's y covers, and loads per span: spans of up
// to kActLoads loads, of equal length.
inline void act8_spans(int64_t d, unsigned* spans, int* per) {
  const int64_t n = (d + kActSpan - 1) / kActSpan;
  *spans = (unsigned)((n + kActLoads - 1) / kActLoads);
  *per = (int)((n + *spans - 1) / *spans);
}

template <class T>
void launch_act8_dequantize(const int8_t* q, const float* scale, int64_t rows, int64_t d, T* out, int64_t ldo,
                            int64_t rows_pad, hipStream_t st) {
  unsigned spans;
  int per;
  act8_spans(ldo, &spans, &per);
  hipLaunchKernelGGL(act8_dequantize_kernel<T>, dim3((unsigned)((rows_pad + kActRows - 1) / kActRows), spans),
                     dim3(64 * kActRows), 0, st, q, scale, (int)((d + kActBlock - 1) / kActBlock), rows, (int)d, per,
                     out, ldo, rows_pad);
}

}  // namespace kd
