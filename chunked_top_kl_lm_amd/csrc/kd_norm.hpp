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
// is held in registers, packed as it was loaded, between its statistics and
// its output, so it is read once and the variance is the two-pass one (no
// cancellation).  Narrow rows belong to one wave (the forward's up to 6 * 512,
// the backward's up to 1024 elements): all reductions are lane exchanges, no
// barrier; wider rows are spread over two to sixteen waves.  131072 bf16 rows
// of 2880 with checkpoints in 8 bits: forward 351 us (1.91 GB, 5.4 TB/s),
// backward 402 us (1.91 GB, 4.7 TB/s) and 5 us for the partial rows, where a
// copy of gigabytes reaches 4.7 (read and write counted); 8192 rows without
// checkpoints 22 and 31 us, what of them the caches hold included.
//
// The weight gradient: each lane owns fixed columns and adds its rows' terms
// in fp32 registers; a block's rows are joined in LDS and a block writes one
// partial row; a second kernel adds the partial rows.  Everything runs in a
// fixed order, so the results are the same bits from call to call.
#pragma once

#include <type_traits>

#include "kd_act8.hpp"

namespace kd {

// Rows per block of threads and its size: WAVES waves (four in the forward;
// eight in the backward, whose blocks write a partial row each), or one row of
// more.
template <int WPR, int WAVES> struct NormCfg {
  static constexpr int kRows = WPR < WAVES ? WAVES / WPR : 1;
  static constexpr int kWaves = WPR * kRows;
  static constexpr int kThreads = 64 * kWaves;
};
template <int WPR> using NormFwdCfg = NormCfg<WPR, 4>;
template <int WPR> using NormBwdCfg = NormCfg<WPR, 8>;

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
      const float2 v = s_red[w / WPR * WPR + i];
      a += v.x;
      b += v.y;
    }
  }
  return make_float2(a, b);
}
// Vectors of a row that every lane holds in each variant (a variant serves
// rows wider than the next narrower one's); of the others a lane may have none.
constexpr int norm_whole(int NV) { return NV == 6 ? 4 : NV == 3 ? 2 : NV / 2; }

// The row's columns: lane vectors of eight up to d8 = d rounded down to a
// multiple of 8, then up to seven single columns that lanes 0 .. tail - 1 of
// one wave hold one each (the wave whose vectors go on there, so that it also
// holds the rest of the last block of an 8-bit checkpoint).  No vector
// crosses the row's end, and the code has one path.
template <int WPR, int NV>
struct NormCols {
  static constexpr int S = 512 * WPR;              // columns per vector of every lane
  int d, d8, tail, c0, lane;
  bool owner;                                      // (uniform per wave) has the tail
  __device__ __forceinline__ explicit NormCols(int d_) : d(d_), d8(d_ & ~7), tail(d_ & 7) {
    lane = threadIdx.x & 63;
    const int wave = (int)(threadIdx.x >> 6) % WPR;
    c0 = 8 * (64 * wave + lane);
    owner = tail > 0 && (d8 / 512) % WPR == wave;
  }
  __device__ __forceinline__ int col(int i) const { return c0 + i * S; }
  __device__ __forceinline__ bool has(int i) const { return i < norm_whole(NV) || col(i) < d8; }
  __device__ __forceinline__ bool has_tail() const { return owner && lane < tail; }
  __device__ __forceinline__ int tail_vec() const { return d8 / S; }          // i of the slot after the last vector
  __device__ __forceinline__ int tail_lane() const { return (d8 / 8) & 63; }  // its lane
  // vector i of a row (zeros where the lane has none), its tail column
  template <class T>
  __device__ __forceinline__ Raw8<T> load(const T* row, int i) const {
    Raw8<T> r = {};
    if (has(i)) r = raw_load8(row + col(i));
    return r;
  }
  template <class T>
  __device__ __forceinline__ float load_tail(const T* row) const {
    return has_tail() ? widen(row[d8 + lane]) : 0.f;
  }
  template <class T>
  __device__ __forceinline__ void store(T* row, int i, const Vec8& v) const {
    if (has(i)) store8(row + col(i), v);
  }
  template <class T>
  __device__ __forceinline__ void store_tail(T* row, float v) const {
    if (has_tail()) narrow(row + d8 + lane, v);
  }
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
__global__ __launch_bounds__(NormFwdCfg<WPR>::kThreads) void norm_fwd_kernel(NormFwdArgs A) {
  __shared__ float2 s_red[2][NormFwdCfg<WPR>::kWaves];
  constexpr int R = NormFwdCfg<WPR>::kRows;
  static_assert(WPR == 1 || R == 1, "rows of one block advance together");
  const NormCols<WPR, NV> C(A.d);
  const int wave = threadIdx.x >> 6, d = A.d;
  // one row per wave (or block) and launch; the loop only serves row counts
  // past the grid's limit
  for (int64_t t = (int64_t)blockIdx.x * R + (R > 1 ? wave : 0); t < A.T; t += (int64_t)gridDim.x * R) {
    const T* xr = (const T*)A.x + t * A.ldx;
    Raw8<T> x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = C.load(xr, i);
    const float xt = C.load_tail(xr);
    float s = xt;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Vec8 v = unpack(x[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v.v[e];
    }
    const float mean = row_sum2<WPR>(s, 0.f, s_red[0]).x / (float)d;
    float m2 = C.has_tail() ? (xt - mean) * (xt - mean) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      keep(x[i]);
      const Vec8 v = unpack(x[i]);
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(v.v[e] - mean, v.v[e] - mean, q);
      m2 += C.has(i) ? q : 0.f;
    }
    const float rstd = 1.f / sqrtf(row_sum2<WPR>(m2, 0.f, s_red[1]).x / (float)d + A.eps);
    T* yr = (T*)A.y + t * (int64_t)d;
    int8_t* qr = CKPT ? A.q + t * (int64_t)d : nullptr;
    float* sr = CKPT ? A.scale + t * A.nb : nullptr;
    uint32_t tail_bits = 0;
    if (CKPT && C.owner)
      tail_bits = read_lane(
          lanes_reduce<8>(__float_as_uint(xt) << 1, [](uint32_t a, uint32_t b) { return max(a, b); }), 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i >= norm_whole(NV) && i * C.S >= d) break;   // uniform: no lane has a column here
      keep(x[i]);
      const Vec8 v = unpack(x[i]);
      if constexpr (CKPT) {
        uint32_t m = block_max16(amax_bits(v));
        if (C.owner && i == C.tail_vec() && (C.tail_lane() ^ C.lane) < 16) m = max(m, tail_bits);
        const float sc = act8_scale(m), inv = 1.f / sc;
        const uint2 w = act8_pack(v, inv);
        const int c = C.col(i);
        if (C.has(i)) __builtin_memcpy(qr + c, &w, 8);
        if ((c & (kActBlock - 1)) == 0 && c < d) sr[c / kActBlock] = sc;
        if (C.owner && i == C.tail_vec()) {
          const float inv_t = read_lane(inv, C.tail_lane());
          if (C.has_tail()) qr[C.d8 + C.lane] = act8_one(xt, inv_t);
        }
      }
      const Vec8 w = unpack(C.load((const WT*)A.w, i));
      Vec8 y;
      if (A.b) {
        const Vec8 b = unpack(C.load((const WT*)A.b, i));
#pragma unroll
        for (int e = 0; e < 8; ++e) y.v[e] = fmaf((v.v[e] - mean) * rstd, w.v[e], b.v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y.v[e] = (v.v[e] - mean) * rstd * w.v[e];
      }
      C.store(yr, i, y);
    }
    if (C.owner)
      C.store_tail(yr, fmaf((xt - mean) * rstd, C.load_tail((const WT*)A.w), A.b ? C.load_tail((const WT*)A.b) : 0.f));
    if (C.lane == 0 && (WPR == 1 || wave == 0)) {
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

// Rows of eight vectors per lane (wider than 16384) are not held in
// registers beside the accumulators: their second pass reads them again from
// the L2.  (Loading the next row ahead of each row's work, for 28 registers
// more, measured slower: 479 against 464 us for the kernel of then, 128K rows of
// 2880 from 8 bits.)
template <int WPR, int NV> constexpr bool norm_hold() { return WPR * NV < 64; }

// Blocks of rows in turn: block b takes rows b, b + grid, ... (times kRows).
template <class T, class WT, int WPR, int NV, bool CKPT>
__global__ __launch_bounds__(NormBwdCfg<WPR>::kThreads, (sizeof(T) == 2 && sizeof(WT) == 2 && NV < 4 ? 4 : 1))
void norm_bwd_kernel(NormBwdArgs A) {
  typedef typename std::conditional<CKPT, int8_t, T>::type XT;
  typedef NormBwdCfg<WPR> Cfg;
  constexpr bool HOLD = norm_hold<WPR, NV>();
  constexpr int R = Cfg::kRows;
  __shared__ float2 s_red[2][Cfg::kWaves];
  __shared__ float s_acc[R > 1 ? 2 * NV * 512 * WPR + 16 : 1];
  const NormCols<WPR, NV> C(A.d);
  const int lane = C.lane, d = A.d;
  // row of the block, wave of the row (uniform per wave)
  const int slot = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) / WPR);
  const int wr = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) % WPR);
  Vec8 aw[NV], ab[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[i].v[e] = ab[i].v[e] = 0.f;
  float awt = 0.f, abt = 0.f;
  int flip = 0;
  const float inv_d = 1.f / (float)d;
  const int64_t ldx = CKPT ? (int64_t)d : A.ldx;
  const XT* xb = CKPT ? (const XT*)A.q : (const XT*)A.x;

  struct Row {
    Raw8<XT> x[NV];
    Raw8<T> dy[NV];
    float sc[NV], mean, rstd, xt, gt;
  };
  auto load_vec = [&](Row& r, int64_t t, int i) {
    r.dy[i] = C.load((const T*)A.dy + t * (int64_t)d, i);
    r.x[i] = C.load(xb + t * ldx, i);
    r.sc[i] = 1.f;
    if constexpr (CKPT) r.sc[i] = C.has(i) ? A.scale[t * A.nb + C.col(i) / kActBlock] : 0.f;
  };
  // (a slot past the last row gets the last row's loads and adds nothing)
  auto load_row = [&](Row& r, int64_t t) {
    r.mean = A.mean[t];
    r.rstd = A.rstd[t];
    if constexpr (HOLD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) load_vec(r, t, i);
    }
    r.xt = r.gt = 0.f;
    if (C.owner) {
      r.gt = C.load_tail((const T*)A.dy + t * (int64_t)d);
      r.xt = C.load_tail(xb + t * ldx);
      if constexpr (CKPT) r.xt *= A.scale[t * A.nb + C.d8 / kActBlock];
    }
  };
  auto row = [&](Row& r, int64_t t, bool live) {
    // xh = x rstd - mean rstd in one step: off by a few roundings of |x| and
    // |mean| over the deviation, as the rounding of mean alone is.  Where a
    // lane has no column, dy and w are zero, so every term below is too.
    const float rstd = r.rstd, shift = -r.mean * rstd;
    auto xhat = [&](int i) {
      Vec8 v = unpack(r.x[i]);
      const float step = CKPT ? r.sc[i] * rstd : rstd;
#pragma unroll
      for (int e = 0; e < 8; ++e) v.v[e] = fmaf(v.v[e], step, shift);
      return v;
    };
    const float xt = C.has_tail() ? fmaf(r.xt, rstd, shift) : 0.f;
    const float wt = C.owner ? C.load_tail((const WT*)A.w) : 0.f;
    float sg = r.gt * wt, sgx = r.gt * wt * xt;
    if (live) {
      awt = fmaf(r.gt, xt, awt);
      abt += r.gt;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (!HOLD) load_vec(r, t, i);
      const Vec8 w = unpack(C.load((const WT*)A.w, i));
      const Vec8 g = unpack(r.dy[i]), xh = xhat(i);
      if (live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          aw[i].v[e] = fmaf(g.v[e], xh.v[e], aw[i].v[e]);
          ab[i].v[e] += g.v[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gw = g.v[e] * w.v[e];
        sg += gw;
        sgx = fmaf(gw, xh.v[e], sgx);
      }
      // one vector at a time: the accumulators and the held rows leave few
      // registers
      settle(aw[i]);
      settle(ab[i]);
      settle(sg, sgx);
      if constexpr (!HOLD) asm volatile("" ::: "memory");        // the next vector's loads stay behind this one
    }
    const float2 m = row_sum2<WPR>(sg, sgx, s_red[flip]);
    flip ^= 1;
    if (A.dx && live) {
      // dx = rstd (dy w) + t, t = -rstd (mean(g) + xh mean(g xh))
      const float mg = -m.x * inv_d * rstd, mgx = -m.y * inv_d * rstd;
      T* dxr = (T*)A.dx + t * (int64_t)d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i >= norm_whole(NV) && i * C.S >= d) break;
        if constexpr (HOLD) {
          keep(r.dy[i]);
          keep(r.x[i]);
        } else {
          load_vec(r, t, i);
        }
        const Vec8 w = unpack(C.load((const WT*)A.w, i));
        const Vec8 g = unpack(r.dy[i]);
        Vec8 o = xhat(i);
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = fmaf(g.v[e] * w.v[e], rstd, fmaf(o.v[e], mgx, mg));
        C.store(dxr, i, o);
        if constexpr (!HOLD) asm volatile("" ::: "memory");
      }
      if (C.owner) C.store_tail(dxr, fmaf(r.gt * wt, rstd, fmaf(xt, mgx, mg)));
    }
  };

  // the block's rows advance together (the barrier of row_sum2)
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t t = (int64_t)blockIdx.x * R;
  auto at = [&](int64_t base) { return min(base + slot, A.T - 1); };
  for (; t < A.T; t += step) {
    Row r;
    load_row(r, at(t));
    row(r, at(t), t + slot < A.T);
  }

  if (!A.part) return;
  float* pw = A.part + (int64_t)blockIdx.x * 2 * d;
  if constexpr (R > 1) {
    // join the slots' columns, in their order
    constexpr int H = NV * 512 * WPR;              // floats per sum
    float* s_tail = s_acc + 2 * H;
    for (int q = 0; q < R; ++q) {
      if (slot == q) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // element e of column group (i, wave, lane) at [i][wave][e][lane]: no bank conflicts
            const int k = ((i * WPR + wr) * 8 + e) * 64 + lane;
            s_acc[k] = q ? s_acc[k] + aw[i].v[e] : aw[i].v[e];
            s_acc[H + k] = q ? s_acc[H + k] + ab[i].v[e] : ab[i].v[e];
          }
        if (C.has_tail()) {
          s_tail[lane] = q ? s_tail[lane] + awt : awt;
          s_tail[8 + lane] = q ? s_tail[8 + lane] + abt : abt;
        }
      }
      __syncthreads();
    }
    for (int k = threadIdx.x >> 6; k < 2 * NV * WPR; k += Cfg::kWaves) {
      Vec8 o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o.v[e] = s_acc[(k * 8 + e) * 64 + lane];
      const int c = 512 * (k % (NV * WPR)) + 8 * lane;
      if (c < C.d8) store8(pw + (k < NV * WPR ? 0 : d) + c, o);
    }
    if (threadIdx.x < 64 && lane < C.tail) {
      pw[C.d8 + lane] = s_tail[lane];
      pw[d + C.d8 + lane] = s_tail[8 + lane];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      C.store(pw, i, aw[i]);
      C.store(pw + d, i, ab[i]);
    }
    C.store_tail(pw, awt);
    C.store_tail(pw + d, abt);
  }
}

// Columns of the partial rows summed in a fixed order: 64 columns per block,
// sixteen waves take every sixteenth partial row, joined in LDS.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* part, int blocks, int d, float* dw, float* db) {
  __shared__ float s[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = blockIdx.x * 64 + lane;
  float a = 0.f;
  if (j < 2 * d) {
    const float* p = part + j;
#pragma unroll 8
    for (int b = wave; b < blocks; b += 16) a += p[(int64_t)b * 2 * d];
  }
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
