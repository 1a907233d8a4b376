// kd_logits.hpp -- head logits z[t, v] = h_t . W_v handed to the caller as
// fp32 [T, V] (what sampling reads).
//
// Many rows: the library's NT GEMM (kd_gemm.hpp), z^T = W H^T, with an
// epilogue that writes row t's logits along v.  Bound by the matrix cores.
//
// Few rows (a decoding step): every element of W is used T times only, so the
// product is bound by reading W once.  skinny_logits_kernel needs no LDS and
// no barrier: a wave owns 16 vocabulary rows, streams them straight from HBM
// into matrix-core operands (v_mfma_f32_16x16x32_bf16: lane l supplies row
// l % 16 and eight consecutive k; fp32: four v_mfma_f32_16x16x4_f32 per
// 16-byte unit) and multiplies each by up to 16 * NT hidden rows, which
// stay in the caches.  Several K steps of loads are issued ahead of their
// products, and thousands of waves keep HBM busy.
#pragma once

#include "kd_gemm.hpp"
#include "kd_rows.hpp"

namespace kd {

// GEMM epilogue: columns 32 j .. + 31 of the wave's tile are staged in its
// share of the freed LDS ring as [32 t][32 FM v] fp32 (16-byte unit u of row
// t at u ^ (t mod units): conflict-free writes and reads) and leave as
// 16-byte stores of whole row segments.  Rows of z start at any multiple of
// 4 bytes; units that cross the end of a row are stored element by element.
struct EpiStoreLogits {
  float* z;       // [N][M]
  int64_t ldz;
  int M, N;       // vocabulary, rows

  template <int FM, int FN>
  __device__ __forceinline__ void apply(f32x16 (&acc)[FM][FN], const EpiCtx& c) const {
    if (c.m0 >= M) return;
    constexpr int U = 8 * FM;                       // 16-byte units per staged row
    constexpr int RPI = 64 / U;                     // rows per read of the wave
    char* lds = c.smem + c.wid * (c.smem_bytes / c.nwaves);
    const int tl = acc_col(c.lane);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if (c.n0 + 32 * j >= N) break;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
          const int u = 8 * i + 2 * g4 + (c.lane >> 5);
          *(f32x4*)(lds + tl * (U * 16) + ((u ^ (tl & (U - 1))) << 4)) =
              f32x4{acc[i][j][4 * g4], acc[i][j][4 * g4 + 1], acc[i][j][4 * g4 + 2], acc[i][j][4 * g4 + 3]};
        }
      __builtin_amdgcn_s_waitcnt(0xC07F);           // lgkmcnt(0): the wave's staging writes are done
      const int u = c.lane & (U - 1);
      const int v = c.m0 + 4 * u;
#pragma unroll
      for (int q = 0; q < 32 / RPI; ++q) {
        const int r = q * RPI + c.lane / U;
        const f32x4 val = *(const f32x4*)(lds + r * (U * 16) + ((u ^ (r & (U - 1))) << 4));
        const int t = c.n0 + 32 * j + r;
        if (t >= N) continue;
        float* o = z + (int64_t)t * ldz + v;
        if (v + 4 <= M) {
          __builtin_memcpy(o, &val, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (v + e < M) o[e] = val[e];
        }
      }
      // the wave's LDS operations run in order: the next half's writes
      // follow this half's reads
      __builtin_amdgcn_s_waitcnt(0xC07F);
    }
  }
};

// One 16-byte unit of a row, elements k .. k + n - 1 (zeros past d).
template <class E>
__device__ __forceinline__ u32x4 unit16(const typename E::T* row, int k, int d) {
  constexpr int n = 16 / E::kBytes;
  u32x4 u = {0, 0, 0, 0};
  if (k + n <= d) {
    __builtin_memcpy(&u, row + k, 16);
  } else if (k < d) {
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (k + i < d) {
        if constexpr (E::kBytes == 2) u[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
        else u[i] = __float_as_uint(row[k + i]);
      }
  }
  return u;
}

template <class E> __device__ __forceinline__ void mfma16_unit(f32x4& acc, u32x4 a, u32x4 b);
template <> __device__ __forceinline__ void mfma16_unit<Bf16>(f32x4& acc, u32x4 a, u32x4 b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0,
                                                0, 0);
}
template <> __device__ __forceinline__ void mfma16_unit<F32>(f32x4& acc, u32x4 a, u32x4 b) {
  const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa.x, fb.x, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa.y, fb.y, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa.z, fb.z, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fa.w, fb.w, acc, 0, 0, 0);
}

constexpr int kSkinnyWaves = 4;    // waves (16 vocabulary rows each) per block
constexpr int kSkinnyAhead = 8;    // K steps of W in flight per wave

// z for up to 16 * NT rows.  Accumulator layout of the 16x16 tiles: register
// r of lane l holds C[4 * (l / 16) + r][l % 16]: four consecutive v of one row t.
template <class E, int NT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_logits_kernel(const typename E::T* H, int64_t ldh, int T,
                                                                          const typename E::T* W, int V, int d,
                                                                          float* z, int64_t ldz) {
  constexpr int kUnit = 16 / E::kBytes;             // elements per lane and K step
  constexpr int kStep = 4 * kUnit;                  // elements of K per step
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int v0 = (blockIdx.x * kSkinnyWaves + wave) * 16;
  if (v0 >= V) return;
  const int row = lane & 15, kl = (lane >> 4) * kUnit;
  const typename E::T* w = W + (int64_t)min(v0 + row, V - 1) * d;
  const typename E::T* h[NT];
  int dh[NT];                                       // rows past T read nothing: zeros
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = 16 * n + row;
    h[n] = H + (int64_t)min(t, T - 1) * ldh;
    dh[n] = t < T ? d : 0;
  }
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  int k = 0;
  for (; k + kSkinnyAhead * kStep <= d; k += kSkinnyAhead * kStep) {
    u32x4 a[kSkinnyAhead];
#pragma unroll
    for (int i = 0; i < kSkinnyAhead; ++i) __builtin_memcpy(&a[i], w + k + i * kStep + kl, 16);
#pragma unroll
    for (int i = 0; i < kSkinnyAhead; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) mfma16_unit<E>(acc[n], a[i], unit16<E>(h[n], k + i * kStep + kl, dh[n]));
  }
  for (; k < d; k += kStep) {
    const u32x4 a = unit16<E>(w, k + kl, d);
#pragma unroll
    for (int n = 0; n < NT; ++n) mfma16_unit<E>(acc[n], a, unit16<E>(h[n], k + kl, dh[n]));
  }
  const int v = v0 + 4 * (lane >> 4);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = 16 * n + row;
    if (t >= T) continue;
    float* o = z + (int64_t)t * ldz + v;
    if (v + 4 <= V) {
      __builtin_memcpy(o, &acc[n], 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v + e < V) o[e] = acc[n][e];
    }
  }
}

}  // namespace kd
