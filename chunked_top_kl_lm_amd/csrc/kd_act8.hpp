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
// four blocks per load, several loads in flight.  fp32 rows of 2880, 32768 of
// them (475 MB a way): 111 us to bytes, 96 us back, 4.3 and 4.9 TB/s where a
// copy of gigabytes reaches 4.7 (read and write counted); 2048 bf16 rows, in
// the caches, 6 us each way.
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
  } else if (c < d) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < d) qrow[c + i] = (int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
  if ((c & (kActBlock - 1)) == 0 && c < d) srow[c / kActBlock] = s;
}

constexpr int kActRows = 4;       // rows (waves) of a block of threads
constexpr int kActSpan = 512;     // elements of a row that a wave takes per load
constexpr int kActLoads = 4;      // most loads per wave, all in flight

// Grid: for each group of kActRows rows, its parts of PER * kActSpan elements
// (neighbouring blocks read neighbouring memory).
template <class T, int PER>
__global__ __launch_bounds__(64 * kActRows) void act8_quantize_kernel(const T* x, int64_t ldx, int64_t rows, int d,
                                                                      int8_t* q, float* scale, int nb, int parts) {
  const int group = blockIdx.x / parts, part = blockIdx.x - group * parts;
  const int64_t t = (int64_t)group * kActRows + (threadIdx.x >> 6);
  if (t >= rows) return;                            // whole waves
  const T* xr = x + t * ldx;
  int8_t* qr = q + t * d;
  float* sr = scale + t * nb;
  const int c0 = part * PER * kActSpan, cl = c0 + 8 * (int)(threadIdx.x & 63);
  Vec8 v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = row_load8(xr, cl + i * kActSpan, d);
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (c0 + i * kActSpan < d) act8_store(v[i], qr, sr, cl + i * kActSpan, d);
}

// Back to x' (rounded to the output's type).  Rows of ldo elements; with
// rows_pad > rows or ldo > d the padding is written with zeros (what the
// matrix products read).
template <class T, int PER>
__global__ __launch_bounds__(64 * kActRows) void act8_dequantize_kernel(const int8_t* q, const float* scale, int nb,
                                                                        int64_t rows, int d, T* out, int64_t ldo,
                                                                        int64_t rows_pad, int parts) {
  const int group = blockIdx.x / parts, part = blockIdx.x - group * parts;
  const int64_t t = (int64_t)group * kActRows + (threadIdx.x >> 6);
  if (t >= rows_pad) return;
  const int dl = t < rows ? d : 0;                  // a padding row has no elements
  const int8_t* qr = q + (t < rows ? t : 0) * d;
  const float* sr = scale + (t < rows ? t : 0) * nb;
  T* o = out + t * ldo;
  const int cl = part * PER * kActSpan + 8 * (int)(threadIdx.x & 63);
  Vec8 v[PER];
  float s[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = cl + i * kActSpan;
    v[i] = row_load8(qr, c, dl);
    s[i] = c < dl ? sr[c / kActBlock] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = cl + i * kActSpan;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i].v[e] *= s[i];
    if (c + 8 > dl && c < dl) {                     // the vector that crosses the row's end: zeros stay zeros
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i].v[e] = c + e < dl ? v[i].v[e] : 0.f;
    }
    row_store8(o, c, (int)ldo, v[i]);
  }
}

// Parts of a row, and loads per part: as few parts
// of up to kActLoads loads as hold the row, of equal length.
inline void act8_parts(int64_t d, unsigned* parts, int* per) {
  const int64_t n = (d + kActSpan - 1) / kActSpan;
  *parts = (unsigned)((n + kActLoads - 1) / kActLoads);
  *per = (int)((n + *parts - 1) / *parts);
}
// One launch covers all rows: its threads are counted in 32 bits.
inline bool act8_fits(int64_t rows, int64_t d) {
  if (rows < 1 || d < 1 || rows > (1ll << 24) || d > (1ll << 24)) return false;
  unsigned parts;
  int per;
  act8_parts(d, &parts, &per);
  return (rows + kActRows - 1) / kActRows * parts < (1ll << 24);
}
inline unsigned act8_groups(int64_t rows) { return (unsigned)((rows + kActRows - 1) / kActRows); }

template <class T>
void launch_act8_quantize(const T* x, int64_t ldx, int64_t rows, int64_t d, int8_t* q, float* scale, hipStream_t st) {
  unsigned parts;
  int per;
  act8_parts(d, &parts, &per);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(act8_groups(rows) * parts), dim3(64 * kActRows), 0, st, x, ldx, rows, (int)d, q,
                       scale, (int)((d + kActBlock - 1) / kActBlock), (int)parts);
  };
  if (per == 1) launch(act8_quantize_kernel<T, 1>);
  else if (per == 2) launch(act8_quantize_kernel<T, 2>);
  else if (per == 3) launch(act8_quantize_kernel<T, 3>);
  else launch(act8_quantize_kernel<T, 4>);
}

template <class T>
void launch_act8_dequantize(const int8_t* q, const float* scale, int64_t rows, int64_t d, T* out, int64_t ldo,
                            int64_t rows_pad, hipStream_t st) {
  unsigned parts;
  int per;
  act8_parts(ldo, &parts, &per);
  auto launch = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(act8_groups(rows_pad) * parts), dim3(64 * kActRows), 0, st, q, scale,
                       (int)((d + kActBlock - 1) / kActBlock), rows, (int)d, out, ldo, rows_pad, (int)parts);
  };
  if (per == 1) launch(act8_dequantize_kernel<T, 1>);
  else if (per == 2) launch(act8_dequantize_kernel<T, 2>);
  else if (per == 3) launch(act8_dequantize_kernel<T, 3>);
  else launch(act8_dequantize_kernel<T, 4>);
}

}  // namespace kd
