// kd_logits.hpp -- head logits z[t, v] = h_t . W_v handed to the caller as
// fp32 [T, V] (what sampling reads).
//
// Many rows: the library's NT GEMM (kd_gemm.hpp), z^T = W H^T, with an
// epilogue that writes row t's logits along v.  Bound by the matrix cores: at
// d = 2880, V = 201088 512 rows take 550 us (1.08 PFLOP/s; a plain product of
// 8192^3 by the vendor's library reaches 1.15 on this card), 2048 2.06 ms.
//
// Few rows (a decoding step): every element of W is used T times only, so the
// product is bound by reading W once.  In skinny_logits_kernel a wave owns 16
// vocabulary rows and streams them from HBM straight into matrix-core operands
// (v_mfma_f32_16x16x32_bf16: lane l supplies row l % 16 and eight consecutive
// k; fp32: four v_mfma_f32_16x16x4_f32 per 16-byte unit), a chunk of 256 bytes
// per row ahead of the products.  The hidden rows' chunk, which all waves need,
// goes through LDS once per block (two buffers, one barrier per chunk).  At d =
// 2880, V = 201088 one row takes 204 us (5.7 TB/s of the 6.0 .. 6.4 that plain
// reads of as much memory reach), 32 rows 234 us; read from the caches by every
// wave instead, the hidden rows made 24 rows of V = 128256 take 280 us, now 145.
#pragma once

#include "kd_gemm.hpp"
#include "kd_rows.hpp"

namespace kd {

// GEMM epilogue: columns 32 j .. + 31 of the wave's tile, up to four 32-row
// tiles at a time, are staged in its share of the freed LDS ring as [32 t][32 B
// v] fp32 (16-byte unit u of row t at u ^ (t mod units): conflict-free writes
// and reads) and leave as 16-byte stores of whole row segments.  Rows of z
// start at any multiple of 4 bytes; units that cross the end of a row are
// stored element by element.
struct EpiStoreLogits {
  float* z;       // [N][M]
  int64_t ldz;
  int M, N;       // vocabulary, rows

  template <int FM, int FN>
  __device__ __forceinline__ void apply(f32x16 (&acc)[FM][FN], const EpiCtx& c) const {
    static_assert(FM <= 5, "one group of four tiles and one more");
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if (c.n0 + 32 * j >= N) break;
      constexpr int B = FM < 4 ? FM : 4;
      store<B, 0>(acc, j, c);
      if constexpr (FM == 5) store<1, 4>(acc, j, c);
    }
  }

  // tiles I0 .. I0 + B - 1 of the wave's rows
  template <int B, int I0, int FM, int FN>
  __device__ __forceinline__ void store(f32x16 (&acc)[FM][FN], int j, const EpiCtx& c) const {
    static_assert(B == 1 || B == 2 || B == 4, "units per staged row");
    constexpr int U = 8 * B;                        // 16-byte units per staged row
    constexpr int RPI = 64 / U;                     // rows per read of the wave
    if (c.m0 + 32 * I0 >= M) return;
    char* lds = c.smem + c.wid * (c.smem_bytes / c.nwaves);
    const int tl = acc_col(c.lane);
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int g4 = 0; g4 < 4; ++g4) {
        const int u = 8 * i + 2 * g4 + (c.lane >> 5);
        const f32x16& a = acc[I0 + i][j];
        *(f32x4*)(lds + tl * (U * 16) + ((u ^ (tl & (U - 1))) << 4)) =
            f32x4{a[4 * g4], a[4 * g4 + 1], a[4 * g4 + 2], a[4 * g4 + 3]};
      }
    __builtin_amdgcn_s_waitcnt(0xC07F);             // lgkmcnt(0): the wave's staging writes are done
    const int u = c.lane & (U - 1);
    const int v = c.m0 + 32 * I0 + 4 * u;
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
    // the wave's LDS operations run in order: the next group's writes follow
    // this group's reads
    __builtin_amdgcn_s_waitcnt(0xC07F);
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

constexpr int kSkinnySteps = 4;    // K steps (64 bytes of a row) per chunk
constexpr int kSkinnyRow = 64 * kSkinnySteps + 16;   // LDS bytes of a hidden row's chunk: a fragment's 16 rows
                                                     // start 4 banks apart and cover all 64

// z for up to 16 * NT rows.  Accumulator layout of the 16x16 tiles: register
// r of lane l holds C[4 * (l / 16) + r][l % 16]: four consecutive v of one row t.
template <class E, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void skinny_logits_kernel(const typename E::T* H, int64_t ldh, int T,
                                                                          const typename E::T* W, int V, int d,
                                                                          float* z, int64_t ldz) {
  constexpr int kUnit = 16 / E::kBytes;             // elements of a 16-byte unit
  constexpr int kStep = 4 * kUnit;                  // of a K step
  constexpr int kChunk = kSkinnySteps * kStep;
  constexpr int kUnits = 4 * kSkinnySteps;          // units of a row's chunk
  constexpr int kStage = 16 * NT * kUnits / (64 * WAVES);   // units staged per thread
  __shared__ __attribute__((aligned(16))) char s_h[2][16 * NT * kSkinnyRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int v0 = (blockIdx.x * WAVES + wave) * 16;
  const int row = lane & 15, ul = lane >> 4;        // fragment row, unit of a step
  const typename E::T* w = W + (int64_t)min(v0 + row, V - 1) * d;
  const int chunks = (d + kChunk - 1) / kChunk;

  u32x4 hs[kStage];
  auto load_h = [&](int c) {
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int q = tid + i * 64 * WAVES, t = q / kUnits, u = q % kUnits;
      hs[i] = unit16<E>(H + (int64_t)min(t, T - 1) * ldh, c * kChunk + u * kUnit, t < T ? d : 0);   // t >= T: zeros
    }
  };
  auto store_h = [&](int c) {
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const int q = tid + i * 64 * WAVES, t = q / kUnits, u = q % kUnits;
      *(u32x4*)(s_h[c & 1] + t * kSkinnyRow + u * 16) = hs[i];
    }
  };
  auto load_w = [&](u32x4 (&a)[kSkinnySteps], int c) {
    if ((c + 1) * kChunk <= d) {                    // uniform
#pragma unroll
      for (int i = 0; i < kSkinnySteps; ++i) __builtin_memcpy(&a[i], w + c * kChunk + i * kStep + ul * kUnit, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kSkinnySteps; ++i) a[i] = unit16<E>(w, c * kChunk + i * kStep + ul * kUnit, d);
    }
  };
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const u32x4 (&a)[kSkinnySteps], int c) {
    const char* h = s_h[c & 1] + row * kSkinnyRow + ul * 16;
#pragma unroll
    for (int i = 0; i < kSkinnySteps; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) mfma16_unit<E>(acc[n], a[i], *(const u32x4*)(h + 16 * n * kSkinnyRow + 64 * i));
  };

  u32x4 a0[kSkinnySteps], a1[kSkinnySteps];
  load_w(a0, 0);
  load_h(0);
  store_h(0);
  __syncthreads();
  // the next chunk's loads are in flight while this one is multiplied; a
  // buffer is rewritten after the barrier that follows its last reads
  for (int c = 0; c < chunks; c += 2) {
    if (c + 1 < chunks) {
      load_w(a1, c + 1);
      load_h(c + 1);
    }
    multiply(a0, c);
    if (c + 1 >= chunks) break;
    store_h(c + 1);
    __syncthreads();
    if (c + 2 < chunks) {
      load_w(a0, c + 2);
      load_h(c + 2);
    }
    multiply(a1, c + 1);
    if (c + 2 < chunks) store_h(c + 2);
    __syncthreads();
  }
  const int v = v0 + 4 * ul;
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
