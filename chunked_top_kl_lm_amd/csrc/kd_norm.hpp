// kd_norm.hpp -- layer norm of rows x [T, d], forward and backward, with the
// input kept for the backward pass as it is or as an 8-bit checkpoint
// (kd_act8.hpp) that the forward kernel writes in the same pass.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) r
//   y  = xh w + b
// and with g = dy w,
//   dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_t dy xh,  db = sum_t dy.
//
// Both are bound by HBM: the forward reads x and writes y, the backward reads
// dy and x (or its bytes) and writes dx; w and b stay in the caches.  A row
// is held in registers between its statistics and its output, so it is read
// once and the variance is the two-pass one (no cancellation).  Rows up to
// kNormWaveMax elements belong to one wave: all reductions are lane exchanges, no
// barrier; wider rows are spread over four or sixteen waves.
//
// The weight gradient: each lane owns fixed columns and adds its rows' terms
// in fp32 registers; a block's waves are joined in LDS and a block writes one
// partial row; a second kernel adds the partial rows.  Everything runs in a
// fixed order, so the results are the same bits from call to call.
#pragma once

#include "kd_act8.hpp"

namespace kd {

// Statistics over a row spread over WPR waves: sums, left in every lane.
// s_red: one float2 per wave of the block, rewritten per call (the caller's
// loop passes alternate halves so that one barrier suffices).
template <int WPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* s_red) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) s_red[w] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      a += s_red[i].x;
      b += s_red[i].y;
    }
  }
  return make_float2(a, b);
}

// Rows per block of threads and its size: four single-wave rows, or one row.
template <int WPR> struct NormCfg {
  static constexpr int kRows = WPR == 1 ? 4 : 1;
  static constexpr int kThreads = 64 * WPR * kRows;
};

struct NormFwdArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  const void* b;       // or NULL
  float eps;
  int64_t T;
  int d, nb;           // nb: scale blocks per row
  void* y;
  float* mean;
  float* rstd;
  int8_t* q;           // or NULL: no checkpoint
  float* scale;
};

template <class T, class WT, int WPR, int NV, bool CKPT>
__global__ __launch_bounds__(NormCfg<WPR>::kThreads) void norm_fwd_kernel(NormFwdArgs A) {
  __shared__ float2 s_red[2][WPR];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  constexpr int R = NormCfg<WPR>::kRows;
  const int d = A.d, c0 = 8 * ((WPR == 1 ? 0 : 64 * wave) + lane);
  // one row per wave (or block) and launch; the loop only serves row counts
  // past the grid's limit
  for (int64_t t = (int64_t)blockIdx.x * R + (R > 1 ? wave : 0); t < A.T; t += (int64_t)gridDim.x * R) {
  const T* xr = (const T*)A.x + t * A.ldx;
  Vec8 x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = row_load8(xr, c0 + i * 512 * WPR, d);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[i].v[e];
  }
  const float mean = row_sum2<WPR>(s, 0.f, s_red[0]).x / (float)d;
  float m2 = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = c0 + i * 512 * WPR + e < d ? x[i].v[e] - mean : 0.f;
      m2 = fmaf(c, c, m2);
    }
  }
  const float rstd = 1.f / sqrtf(row_sum2<WPR>(m2, 0.f, s_red[1]).x / (float)d + A.eps);
  T* yr = (T*)A.y + t * (int64_t)d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * 512 * WPR;
    if (i * 512 * WPR >= d) break;                 // uniform: no lane has a column here
    if constexpr (CKPT) act8_store(x[i], A.q + t * (int64_t)d, A.scale + t * A.nb, c, d);
    const Vec8 w = row_load8((const WT*)A.w, c, d);
    Vec8 y;
    if (A.b) {
      const Vec8 b = row_load8((const WT*)A.b, c, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) y.v[e] = fmaf((x[i].v[e] - mean) * rstd, w.v[e], b.v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y.v[e] = (x[i].v[e] - mean) * rstd * w.v[e];
    }
    row_store8(yr, c, d, y);
  }
  if (lane == 0 && (WPR == 1 || wave == 0)) {
    A.mean[t] = mean;
    A.rstd[t] = rstd;
  }
  }
}

struct NormBwdArgs {
  const void* dy;
  const void* x;       // the input, or NULL with
  const int8_t* q;     // its checkpoint
  const float* scale;
  const void* w;
  const float* mean;
  const float* rstd;
  int64_t ldx, T;
  int d, nb;
  void* dx;            // or NULL
  float* part;         // [blocks][2][d] partial dw and db, or NULL
};

// Blocks of rows in turn: block b takes rows b, b + grid, ... (times kRows).
template <class T, class WT, int WPR, int NV, bool CKPT>
__global__ __launch_bounds__(NormCfg<WPR>::kThreads) void norm_bwd_kernel(NormBwdArgs A) {
  __shared__ float2 s_red[2][WPR];
  __shared__ float s_acc[WPR == 1 ? 2 * NV * 512 : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int d = A.d, c0 = 8 * ((WPR == 1 ? 0 : 64 * wave) + lane);
  constexpr int R = NormCfg<WPR>::kRows;
  Vec8 aw[NV], ab[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[i].v[e] = ab[i].v[e] = 0.f;
  int flip = 0;
  const float inv_d = 1.f / (float)d;
  for (int64_t t = (int64_t)blockIdx.x * R + (R > 1 ? wave : 0); t < A.T; t += (int64_t)gridDim.x * R) {
    const float mean = A.mean[t], rstd = A.rstd[t];
    Vec8 x[NV], dy[NV];
    const T* dyr = (const T*)A.dy + t * (int64_t)d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * 512 * WPR;
      dy[i] = row_load8(dyr, c, d);
      if constexpr (CKPT) x[i] = row_load8(A.q + t * (int64_t)d, c, d);
      else x[i] = row_load8((const T*)A.x + t * A.ldx, c, d);
    }
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * 512 * WPR;
      float sc = 1.f;
      if constexpr (CKPT) sc = c < d ? A.scale[t * A.nb + c / kActBlock] : 0.f;
      const Vec8 w = row_load8((const WT*)A.w, c, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // columns past d: dy and w are zero there, so every term below is too
        const float xe = CKPT ? x[i].v[e] * sc : x[i].v[e];
        const float xh = c + e < d ? (xe - mean) * rstd : 0.f;
        x[i].v[e] = xh;
        aw[i].v[e] = fmaf(dy[i].v[e], xh, aw[i].v[e]);
        ab[i].v[e] += dy[i].v[e];
        const float g = dy[i].v[e] * w.v[e];
        dy[i].v[e] = g;
        sg += g;
        sgx = fmaf(g, xh, sgx);
      }
    }
    const float2 m = row_sum2<WPR>(sg, sgx, s_red[flip]);
    flip ^= 1;
    if (A.dx) {
      const float mg = m.x * inv_d, mgx = m.y * inv_d;
      T* dxr = (T*)A.dx + t * (int64_t)d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        Vec8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = rstd * (dy[i].v[e] - mg - x[i].v[e] * mgx);
        row_store8(dxr, c0 + i * 512 * WPR, d, o);
      }
    }
  }
  if (!A.part) return;
  float* pw = A.part + (int64_t)blockIdx.x * 2 * d;
  if constexpr (WPR == 1) {
    // join the four waves' columns, in the order of the waves
    for (int w = 0; w < 4; ++w) {
      if (wave == w) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // element e of column group (i, lane) at [i][e][lane]: no bank conflicts
            const int at = (i * 8 + e) * 64 + lane;
            s_acc[at] = w ? s_acc[at] + aw[i].v[e] : aw[i].v[e];
            s_acc[NV * 512 + at] = w ? s_acc[NV * 512 + at] + ab[i].v[e] : ab[i].v[e];
          }
      }
      __syncthreads();
    }
    for (int i = wave; i < 2 * NV; i += 4) {
      Vec8 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o.v[e] = s_acc[(i * 8 + e) * 64 + lane];
      row_store8(pw + (i < NV ? 0 : d), 512 * (i < NV ? i : i - NV) + 8 * lane, d, o);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      row_store8(pw, c0 + i * 512 * WPR, d, aw[i]);
      row_store8(pw + d, c0 + i * 512 * WPR, d, ab[i]);
    }
  }
}

// Columns of the partial rows summed in a fixed order: 64 columns per block,
// sixteen waves take every sixteenth partial row, joined in LDS.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* part, int blocks, int d, float* dw, float* db) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = blockIdx.x * 64 + lane;
  float a = 0.f;
  if (j < 2 * d)
    for (int b = wave; b < blocks; b += 16) a += part[(int64_t)b * 2 * d + j];
  s[wave][lane] = a;
  __syncthreads();
  if (wave == 0 && j < 2 * d) {
#pragma unroll
    for (int w = 1; w < 16; ++w) a += s[w][lane];
    if (j < d) {
      if (dw) dw[j] = a;
    } else if (db) {
      db[j - d] = a;
    }
  }
}

}  // namespace kd
