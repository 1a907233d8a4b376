// kd_sample.hpp -- one token id per row of logits z [R, V], from a uniform
// number given per row.
//
// Per row, with temperature T, m the largest logit and w_v = exp((z_v - m)/T):
// the ids are ordered by (z descending, id ascending); the first top_k stay;
// of these the shortest prefix whose mass reaches top_p of theirs; of these
// the ids with w_v >= min_p.  The drawn id is the first, in id order, whose
// inclusive mass exceeds u times the kept mass.
//
// Borders between ids are decided in 64 bits.  w is a double (a polynomial of
// degree 12, relative error about 1e-14 with its argument's rounding), and
// masses are sums of 64-bit integers, W_v = rint(w_v 2^s) with s = 62 -
// ceil(log2 V) (at most 52): integer sums are exact and do not depend on
// their order, so LDS atomics keep the result the same from call to call.
// An id more than 32 T below the largest logit (w < 1.3e-14) has W = 0.
// NaN and -inf logits have no mass; a +inf logit is the largest and shares
// the mass with its equals only.
//
// Bound by HBM: R V e bytes read once.  sample_scan_kernel makes that one
// pass with all of the chip: per 64 ids the largest logit and, where the mass
// of a whole row is needed, per 1024 ids the mass relative to the tile's own
// largest logit.  sample_pick_kernel (one block per row) then reads back
// only the 64-id groups that can hold kept ids: ids are put in 2047 bins of
// T/64 below m, and the groups' maxima say how deep the list must go.  Rows
// whose kept set is too long for a list (a flat row under top_p) are
// streamed again: a histogram of mass over the bins, the one bin at the
// border sorted, then the tiles' kept masses.
#pragma once

#include "kd_layout.hpp"
#include "kd_order.hpp"
#include "kd_rows.hpp"

namespace kd {

constexpr int kSampleBins = 2048;     // bins of T/64 below the largest logit; the last holds the rest
constexpr int kSampleList = 4096;     // longest candidate list (LDS)
constexpr int kSamplePick = 1024;     // threads per row
constexpr int kSampleTopGroups = 512; // top_p alone: groups whose maxima bound the first list

struct SampleArgs {
  const void* z;
  int64_t ldz;
  int R, V;
  const void* u;                      // float or double per row
  int u_is_f64;
  double temperature, top_p, min_p;   // used where the row arrays are NULL
  int top_k;
  const double* temperature_rows;
  const int32_t* top_k_rows;
  const double* top_p_rows;
  const double* min_p_rows;
  float* gmax;                        // [R][groups]
  double* tmass;                      // [R][tiles]
  int groups, tiles;
  int32_t* token;
  float* logprob;                     // or NULL
};

// A row's parameters: values of a row array outside their range mean "off"
// (top_k < 1 or >= V; top_p >= 1 or NaN; min_p <= 0 or NaN) or the strictest
// setting (temperature <= 0 or NaN: the largest logit; top_p <= 0: the first
// id; min_p > 1: w = 1 only).
struct SampleRow {
  double c;          // log2(e) / T
  float cb;          // 64 / T
  double top_p, min_p;
  int top_k;         // 0: off
  bool greedy;
};
__device__ __forceinline__ SampleRow sample_row(const SampleArgs& A, int r) {
  SampleRow p;
  const double t = A.temperature_rows ? A.temperature_rows[r] : A.temperature;
  const int k = A.top_k_rows ? A.top_k_rows[r] : A.top_k;
  const double tp = A.top_p_rows ? A.top_p_rows[r] : A.top_p;
  const double mp = A.min_p_rows ? A.min_p_rows[r] : A.min_p;
  p.top_k = k >= 1 && k < A.V ? k : 0;
  p.top_p = tp < 1.0 ? tp : 1.0;
  p.min_p = mp > 0.0 ? (mp < 1.0 ? mp : 1.0) : 0.0;
  p.greedy = !(t > 0.0) || p.top_k == 1 || p.top_p <= 0.0;
  p.c = 1.4426950408889634 / t;
  p.cb = (float)(64.0 / t);
  return p;
}
// The mass of the whole row is needed: no top_k, and not min_p alone.
__device__ __forceinline__ bool sample_needs_mass(const SampleRow& p) {
  return !p.greedy && p.top_k == 0 && (p.top_p < 1.0 || p.min_p == 0.0);
}

// A logit as the operator sees it: NaN as -inf, -0 as +0.
__device__ __forceinline__ float sample_logit(float x) { return x == x ? x + 0.f : -INFINITY; }

// w = 2^((l - m) c).  2^f on |f| <= 1/2 by its Taylor series in f ln 2 up to
// degree 12 (remainder 0.3466^13 / 13! < 2e-16).
__device__ __forceinline__ double sample_weight(float l, float m, double c) {
  const double y0 = ((double)l - (double)m) * c;
  const double y = y0 > -64.0 ? y0 : -64.0;        // also NaN (inf - inf, inf * 0)
  const double k = rint(y);
  const double f = (y - k) * 0.6931471805599453;
  double p = 1.0 / 479001600.0;
  p = fma(p, f, 1.0 / 39916800.0);
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  // times 2^k, k in [-64, 0], p in [0.7, 1.42]: the exponent field directly
  const double w = __longlong_as_double(__double_as_longlong(p) + (long long)(int)k * (1ll << 52));
  return l == m ? 1.0 : (y0 > -64.0 ? w : 0.0);
}
// Bin of a logit: non-increasing in l.  The last bin has no mass.
__device__ __forceinline__ int sample_bin(float l, float m, float cb) {
  const float x = fminf((m - l) * cb, (float)(kSampleBins - 1));   // NaN (inf * 0): the last bin
  return l == m ? 0 : (l == -INFINITY ? kSampleBins - 1 : (int)x);
}

// Eight or four consecutive logits of a row (-inf past its end).
template <class E> struct SampleVec;
template <> struct SampleVec<Bf16> { static constexpr int N = 8; };
template <> struct SampleVec<F32> { static constexpr int N = 4; };
template <class E>
__device__ __forceinline__ void sample_load(const typename E::T* row, int v, int V, float (&x)[SampleVec<E>::N]) {
  constexpr int N = SampleVec<E>::N;
  if (v + N <= V) {
    u32x4 u;
    __builtin_memcpy(&u, row + v, 16);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (N == 8) x[i] = __uint_as_float((i & 1) ? (u[i >> 1] & 0xffff0000u) : (u[i >> 1] << 16));
      else x[i] = __uint_as_float(u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v + i < V ? load_elem<E>(row + v + i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = sample_logit(x[i]);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
template <class T>
__device__ __forceinline__ T wave_add(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <class T>
__device__ __forceinline__ T wave_incl_scan(T v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const T u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Grid: for each row, its groups of 4 tiles.
template <class E>
__global__ __launch_bounds__(256) void sample_scan_kernel(SampleArgs A) {
  constexpr int N = SampleVec<E>::N, L = 16 / N;   // vectors per lane
  constexpr int LG = kSampleGroup / N;             // lanes that share a group
  const int quads = (A.tiles + 3) / 4;
  const int r = blockIdx.x / quads, lane = threadIdx.x & 63;
  const int tile = (blockIdx.x - r * quads) * 4 + (threadIdx.x >> 6);
  if (tile >= A.tiles) return;
  const typename E::T* row = (const typename E::T*)A.z + (int64_t)r * A.ldz;
  float x[L][N];
#pragma unroll
  for (int j = 0; j < L; ++j) sample_load<E>(row, tile * kSampleTile + j * 64 * N + lane * N, A.V, x[j]);
  const SampleRow p = sample_row(A, r);
  float tm = -INFINITY;
#pragma unroll
  for (int j = 0; j < L; ++j) {
    float g = x[j][0];
#pragma unroll
    for (int i = 1; i < N; ++i) g = fmaxf(g, x[j][i]);
#pragma unroll
    for (int o = 1; o < LG; o <<= 1) g = fmaxf(g, __shfl_xor(g, o));
    const int gi = tile * (kSampleTile / kSampleGroup) + j * (64 / LG) + lane / LG;
    if (lane % LG == 0 && gi < A.groups) A.gmax[(int64_t)r * A.groups + gi] = g;
    tm = fmaxf(tm, g);
  }
  if (!sample_needs_mass(p)) return;
  tm = wave_max(tm);
  double s = 0.0;
  if (tm > -INFINITY) {
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) s += sample_weight(x[j][i], tm, p.c);
  }
  s = wave_add(s);
  if (lane == 0) A.tmass[(int64_t)r * A.tiles + tile] = s;
}

// ---------------------------------------------------------------------------
// One block per row.
// ---------------------------------------------------------------------------
struct SampleShared {
  uint64_t key[kSampleList];       // candidates: cand_key(z, id)
  uint64_t aux[kSampleList];       // group lists; masses; keys by id
  uint64_t hist[kSampleBins];
  uint64_t wsum[16];
  float wmax[16];
  int n, n2, pos;
  uint64_t a, b;
};

__device__ __forceinline__ float block_max(SampleShared& s, float v) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) s.wmax[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s.wmax[0];
#pragma unroll
  for (int i = 1; i < kSamplePick / 64; ++i) v = fmaxf(v, s.wmax[i]);
  __syncthreads();
  return v;
}
// Inclusive prefix sum over the block's threads; total in `total`.
__device__ __forceinline__ uint64_t block_scan(SampleShared& s, uint64_t v, uint64_t& total) {
  const int w = threadIdx.x >> 6;
  v = wave_incl_scan(v);
  if ((threadIdx.x & 63) == 63) s.wsum[w] = v;
  __syncthreads();
  uint64_t add = 0, t = 0;
#pragma unroll
  for (int i = 0; i < kSamplePick / 64; ++i) {
    if (i < w) add += s.wsum[i];
    t += s.wsum[i];
  }
  __syncthreads();
  total = t;
  return v + add;
}
__device__ __forceinline__ double block_sum(SampleShared& s, double v) {
  v = wave_add(v);
  if ((threadIdx.x & 63) == 0) s.wsum[threadIdx.x >> 6] = (uint64_t)__double_as_longlong(v);
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kSamplePick / 64; ++i) v += __longlong_as_double((long long)s.wsum[i]);
  __syncthreads();
  return v;
}

// The first position, in order, whose inclusive prefix of n values reaches
// `target` >= 1 (-1: none), and the prefix before it; value(i) is called once
// per position, in chunks of the block's size.
template <class F>
__device__ __forceinline__ int block_find(SampleShared& s, int n, uint64_t target, F value, uint64_t& before) {
  uint64_t base = 0;
  for (int i0 = 0; i0 < n; i0 += kSamplePick) {
    const int i = i0 + (int)threadIdx.x;
    const uint64_t v = i < n ? value(i) : 0;
    uint64_t total;
    const uint64_t incl = base + block_scan(s, v, total);
    if (base + total >= target) {                  // uniform
      if (incl >= target && incl - v < target) {   // exactly one thread
        s.pos = i;
        s.a = incl - v;
      }
      __syncthreads();
      const int pos = s.pos;
      before = s.a;
      __syncthreads();
      return pos;
    }
    base += total;
  }
  before = base;
  return -1;
}

__device__ __forceinline__ int pow2_at_least(int n) {
  int m = 1;
  while (m < n) m <<= 1;
  return m;
}
__device__ __forceinline__ int key_id(uint64_t k) { return (int)(0xffffffffu - (uint32_t)k); }
__device__ __forceinline__ float key_logit(uint64_t k) { return fkey_inv((uint32_t)(k >> 32)); }

// Sort s.key[0, n) descending (padding to a power of two with zeros).
__device__ __forceinline__ void sort_keys(uint64_t* key, int n) {
  const int m = pow2_at_least(n);
  for (int i = n + (int)threadIdx.x; i < m; i += kSamplePick) key[i] = 0;
  __syncthreads();
  bitonic_desc(key, m);
}

template <class E>
struct SamplePicker {
  typedef typename E::T T;
  static constexpr int N = SampleVec<E>::N;
  const SampleArgs& A;
  SampleShared& s;
  const int r;
  const SampleRow p;
  const T* row;
  const float* gmax;
  uint64_t* tsum;              // the row's tile sums (in place of its tile masses)
  float m;
  double scale;                // 2^s

  __device__ SamplePicker(const SampleArgs& a, SampleShared& sh)
      : A(a), s(sh), r(blockIdx.x), p(sample_row(a, blockIdx.x)), row((const T*)a.z + (int64_t)blockIdx.x * a.ldz),
        gmax(a.gmax + (int64_t)blockIdx.x * a.groups), tsum((uint64_t*)(a.tmass + (int64_t)blockIdx.x * a.tiles)) {
    int sh_bits = 62 - (32 - __clz(max(A.V - 1, 1)));
    sh_bits = min(sh_bits, 52);
    scale = (double)(1ull << sh_bits);
  }
  __device__ __forceinline__ uint64_t mass(float l) const {
    return sample_bin(l, m, p.cb) < kSampleBins - 1 ? (uint64_t)rint(sample_weight(l, m, p.c) * scale) : 0;
  }
  __device__ __forceinline__ double u() const {
    return A.u_is_f64 ? ((const double*)A.u)[r] : (double)((const float*)A.u)[r];
  }
  // The smallest inclusive prefix that exceeds u * total (1 .. total).
  __device__ __forceinline__ uint64_t draw_target(uint64_t total) const {
    const double x = floor(u() * (double)total);
    if (!(x > 0.0)) return 1;                      // also a NaN
    return x >= (double)total ? total : min((uint64_t)x + 1, total);
  }
  __device__ __forceinline__ void emit(int id, float l, uint64_t total) const {
    if (threadIdx.x == 0) {
      A.token[r] = id;
      // ln w of the drawn id minus the ln of the kept mass
      if (A.logprob) A.logprob[r] = (float)((l == m ? 0.0 : ((double)l - (double)m) * p.c * 0.6931471805599453) -
                                            log((double)total / scale));
    }
  }

  // Lowest id of the largest logit.
  __device__ void pick_greedy() {
    int g = A.groups;
    for (int i = threadIdx.x; i < A.groups; i += kSamplePick)
      if (gmax[i] == m) { g = i; break; }
    g = (int)-block_max(s, -(float)g);             // < 2^24: exact
    if (threadIdx.x < 64) {
      const int v = g * kSampleGroup + (int)threadIdx.x;
      const bool hit = v < A.V && sample_logit(load_elem<E>(row + v)) == m;
      const unsigned long long b = __ballot(hit);
      if (threadIdx.x == 0) {
        A.token[r] = g * kSampleGroup + (int)__builtin_ctzll(b);
        if (A.logprob) A.logprob[r] = 0.f;
      }
    }
  }

  // Bin that `want` groups have their maxima in or above (the last one with
  // mass if there are fewer).
  __device__ int group_bin(int want) {
    for (int i = threadIdx.x; i < kSampleBins; i += kSamplePick) s.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < A.groups; i += kSamplePick)
      atomicAdd((unsigned long long*)&s.hist[sample_bin(gmax[i], m, p.cb)], 1ull);
    __syncthreads();
    uint64_t before;
    const int b = block_find(s, kSampleBins - 1, (uint64_t)want, [&](int i) { return s.hist[i]; }, before);
    return b < 0 ? kSampleBins - 2 : b;
  }

  // All ids in bins <= b into s.key (unordered); their number, or a number
  // past kSampleList if they do not fit.
  __device__ int gather(int b) {
    int* list = (int*)s.aux;                       // groups to read: 2 * kSampleList places
    if (threadIdx.x == 0) s.n = s.n2 = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < A.groups; i += kSamplePick)
      if (sample_bin(gmax[i], m, p.cb) <= b) {
        const int at = atomicAdd(&s.n2, 1);
        if (at < 2 * kSampleList) list[at] = i;
      }
    __syncthreads();
    const int ng = s.n2;
    if (ng > kSampleList) return kSampleList + 1;  // at least one id each
    const int lane = threadIdx.x & 63;
    for (int g0 = (threadIdx.x >> 6) * 4; g0 < ng; g0 += 4 * (kSamplePick / 64)) {
      float x[4];
      int v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = g0 + j < ng ? list[g0 + j] * kSampleGroup + lane : A.V;
        x[j] = v[j] < A.V ? sample_logit(load_elem<E>(row + v[j])) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v[j] < A.V && sample_bin(x[j], m, p.cb) <= b) {
          const int at = atomicAdd(&s.n, 1);
          if (at < kSampleList) s.key[at] = cand_key(x[j], (uint32_t)v[j]);
        }
    }
    __syncthreads();
    return s.n;
  }

  // Draw from the list's first n entries whose mass counts: sort by id, find.
  // keep(i) says whether entry i of s.key is kept.
  template <class F>
  __device__ void draw_list(int n, F keep) {
    // aux: (~id, position) keys, largest first = lowest id first
    for (int i = threadIdx.x; i < n; i += kSamplePick)
      s.aux[i] = keep(i) ? (((uint64_t)(uint32_t)s.key[i]) << 32) | (uint32_t)i : 0;
    __syncthreads();
    sort_keys(s.aux, n);
    // entries that are not kept sort last with key 0 and have no mass
    auto value = [&](int i) -> uint64_t {
      const uint64_t a = s.aux[i];
      return a ? mass(key_logit(s.key[(uint32_t)a])) : 0;
    };
    uint64_t total = 0, before;
    for (int i0 = 0; i0 < n; i0 += kSamplePick) {
      const int i = i0 + (int)threadIdx.x;
      uint64_t t;
      block_scan(s, i < n ? value(i) : 0, t);
      total += t;
    }
    const int at = block_find(s, n, draw_target(total), value, before);
    const uint64_t k = s.key[(uint32_t)s.aux[max(at, 0)]];
    emit(key_id(k), key_logit(k), total);
  }

  // Mass of the whole row, in units of 1 / scale, from the scan's tile masses
  // (each relative to its tile's own largest logit).
  __device__ double tile_mass(int i) const {
    float tm = -INFINITY;
    const int g0 = i * (kSampleTile / kSampleGroup);
    for (int g = g0; g < min(g0 + kSampleTile / kSampleGroup, A.groups); ++g) tm = fmaxf(tm, gmax[g]);
    if (!(tm > -INFINITY)) return 0.0;
    return __longlong_as_double((long long)tsum[i]) * sample_weight(tm, m, p.c) * scale;
  }

  // ---- rows whose kept set has no short list -------------------------------
  // Calls f(id, logit) for every id of the row, each thread a strided share.
  template <class F>
  __device__ __forceinline__ void for_row(F f) {
    for (int v = (int)threadIdx.x * N; v < A.V; v += kSamplePick * N * 2) {
      float x[2][N];
      const int v2 = v + kSamplePick * N;
      sample_load<E>(row, v, A.V, x[0]);
      if (v2 < A.V) sample_load<E>(row, v2, A.V, x[1]);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (v + i < A.V) f(v + i, x[0][i]);
      if (v2 < A.V) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (v2 + i < A.V) f(v2 + i, x[1][i]);
      }
    }
  }

  // Tighten `lim` (kept: cand_key >= lim) to the shortest prefix, in
  // descending order, of the kept ids with mass whose count (MASS false) or
  // mass reaches a target; target(total) gives it from their total.
  template <bool MASS, class F>
  __device__ uint64_t cut(uint64_t lim, F target) {
    for (int i = threadIdx.x; i < kSampleBins; i += kSamplePick) s.hist[i] = 0;
    __syncthreads();
    for_row([&](int v, float l) {
      const int b = sample_bin(l, m, p.cb);
      if (b < kSampleBins - 1 && cand_key(l, (uint32_t)v) >= lim)
        atomicAdd((unsigned long long*)&s.hist[b], MASS ? (unsigned long long)mass(l) : 1ull);
    });
    __syncthreads();
    uint64_t total = 0;
    for (int i0 = 0; i0 < kSampleBins; i0 += kSamplePick) {
      uint64_t t;
      block_scan(s, s.hist[i0 + threadIdx.x], t);
      total += t;
    }
    const uint64_t want = target(total);
    uint64_t before;
    const int b = block_find(s, kSampleBins - 1, want, [&](int i) { return s.hist[i]; }, before);
    if (b < 0) return lim;                         // the target is not reached: all stay
    const uint64_t rest = want - before;
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    for_row([&](int v, float l) {
      const uint64_t k = cand_key(l, (uint32_t)v);
      if (sample_bin(l, m, p.cb) == b && k >= lim) {
        const int at = atomicAdd(&s.n, 1);
        if (at < kSampleList) s.key[at] = k;
      }
    });
    __syncthreads();
    const int n = s.n;
    __syncthreads();
    if (n <= kSampleList) {
      sort_keys(s.key, n);
      const int at = block_find(
          s, n, rest, [&](int i) -> uint64_t { return MASS ? mass(key_logit(s.key[i])) : 1; }, before);
      const uint64_t k = s.key[at < 0 ? n - 1 : at];
      __syncthreads();
      return k;
    }
    // more ids in one bin than the list holds (equal logits, mostly): the
    // key at the border digit by digit, a pass over the row per digit
    uint64_t prefix = 0, mask = 0, left = rest;
    for (int shift = 56; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSamplePick) s.hist[i] = 0;
      __syncthreads();
      for_row([&](int v, float l) {
        const uint64_t k = cand_key(l, (uint32_t)v);
        if (sample_bin(l, m, p.cb) == b && k >= lim && (k & mask) == prefix)
          atomicAdd((unsigned long long*)&s.hist[255 - ((k >> shift) & 255)], MASS ? (unsigned long long)mass(l) : 1ull);
      });
      __syncthreads();
      const int at = block_find(s, 256, left, [&](int i) { return s.hist[i]; }, before);
      prefix |= (uint64_t)(255 - max(at, 0)) << shift;
      mask |= 255ull << shift;
      left -= before;
      __syncthreads();
    }
    return prefix;
  }

  // Draw from the ids with cand_key >= lim and w >= min_p, whose masses per
  // tile are in tsum (already, or counted here).
  __device__ void draw_row(uint64_t lim, bool counted) {
    const int lane = threadIdx.x & 63;
    auto kept = [&](int v, float l) -> uint64_t {
      if (v >= A.V || cand_key(l, (uint32_t)v) < lim) return 0;
      if (p.min_p > 0.0 && !(sample_weight(l, m, p.c) >= p.min_p)) return 0;
      return mass(l);
    };
    if (!counted) {
      for (int t = threadIdx.x >> 6; t < A.tiles; t += kSamplePick / 64) {
        uint64_t a = 0;
#pragma unroll
        for (int j = 0; j < 16 / N; ++j) {
          float x[N];
          const int v = t * kSampleTile + j * 64 * N + lane * N;
          sample_load<E>(row, v, A.V, x);
#pragma unroll
          for (int i = 0; i < N; ++i) a += kept(v + i, x[i]);
        }
        a = wave_add(a);
        if (lane == 0) tsum[t] = a;
      }
      __syncthreads();
    }
    uint64_t total = 0, before = 0;
    for (int i0 = 0; i0 < A.tiles; i0 += kSamplePick) {
      const int i = i0 + (int)threadIdx.x;
      uint64_t t;
      block_scan(s, i < A.tiles ? tsum[i] : 0, t);
      total += t;
    }
    const uint64_t want = draw_target(total);
    const int tile = block_find(s, A.tiles, want, [&](int i) { return tsum[i]; }, before);
    if (tile < 0 || threadIdx.x >= 64) return;
    // inside the tile: 16 consecutive ids per lane
    uint64_t w[16], a = 0;
    const int v0 = tile * kSampleTile + lane * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int v = v0 + i;
      const float l = v < A.V ? sample_logit(load_elem<E>(row + v)) : -INFINITY;
      w[i] = kept(v, l);
      a += w[i];
    }
    const uint64_t incl = wave_incl_scan(a);
    uint64_t run = before + incl - a;
    int found = -1, last = -1;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      run += w[i];
      if (w[i]) last = v0 + i;
      if (found < 0 && run >= want && w[i]) found = v0 + i;
    }
    // the lowest lane that reached it; if rounding of the tile's mass left
    // none, the tile's last id with mass
    const unsigned long long hit = __ballot(found >= 0), any = __ballot(last >= 0);
    const int src = hit ? (int)__builtin_ctzll(hit) : (any ? 63 - (int)__builtin_clzll(any) : 0);
    const int id = __shfl(hit ? found : last, src);
    if (id >= 0) emit(id, sample_logit(load_elem<E>(row + id)), total);
  }

  __device__ void pick() {
    float x = -INFINITY;
    for (int i = threadIdx.x; i < A.groups; i += kSamplePick) x = fmaxf(x, gmax[i]);
    m = block_max(s, x);
    if (m == -INFINITY) {                          // nothing to draw from
      if (threadIdx.x == 0) {
        A.token[r] = -1;
        if (A.logprob) A.logprob[r] = -INFINITY;
      }
      return;
    }
    if (p.greedy) return pick_greedy();
    const bool filtered = p.top_k > 0 || p.top_p < 1.0 || p.min_p > 0.0;
    if (!filtered) {
      for (int i = threadIdx.x; i < A.tiles; i += kSamplePick) tsum[i] = (uint64_t)rint(tile_mass(i));
      __syncthreads();
      return draw_row(0, true);
    }
    double row_mass = 0.0;
    if (sample_needs_mass(p)) {
      for (int i = threadIdx.x; i < A.tiles; i += kSamplePick) row_mass += tile_mass(i);
      row_mass = block_sum(s, row_mass);
    }
    // how deep the list must go
    int b = kSampleBins - 2;
    if (p.top_k > 0) b = group_bin(p.top_k);
    else if (p.top_p < 1.0) b = group_bin(kSampleTopGroups);
    // (top_p of top_k's ids needs the mass of all of them)
    if (p.min_p > 0.0 && !(p.top_k > 0 && p.top_p < 1.0)) b = min(b, (int)fmin(-64.0 * log(p.min_p) + 2.0, (double)(kSampleBins - 2)));
    const int n = gather(b);
    if (n <= kSampleList) {
      if (p.top_k == 0 && p.top_p == 1.0)
        return draw_list(n, [&](int i) { return sample_weight(key_logit(s.key[i]), m, p.c) >= p.min_p; });
      sort_keys(s.key, n);
      const int n1 = p.top_k > 0 ? min(n, p.top_k) : n;
      int n2 = n1;
      bool whole = true;
      if (p.top_p < 1.0) {
        double all = row_mass;
        auto value = [&](int i) { return mass(key_logit(s.key[i])); };
        uint64_t total = 0, before;
        for (int i0 = 0; i0 < n1; i0 += kSamplePick) {
          const int i = i0 + (int)threadIdx.x;
          uint64_t t;
          block_scan(s, i < n1 ? value(i) : 0, t);
          total += t;
        }
        if (p.top_k > 0) all = (double)total;
        const double need = fmax(ceil(p.top_p * all), 1.0);
        whole = p.top_k > 0 || (double)total >= need || b == kSampleBins - 2 || cut_by_min_p(b);
        if (whole) {
          const int at = block_find(s, n1, (uint64_t)need, value, before);
          n2 = at < 0 ? n1 : at + 1;
        }
      }
      if (whole)
        return draw_list(n2, [&](int i) {
          return p.min_p == 0.0 || sample_weight(key_logit(s.key[i]), m, p.c) >= p.min_p;
        });
    }
    // the kept set by streaming the row
    uint64_t lim = 0;
    if (p.top_k > 0) lim = cut<false>(lim, [&](uint64_t) { return (uint64_t)p.top_k; });
    if (p.top_p < 1.0)
      lim = cut<true>(lim, [&](uint64_t total) { return (uint64_t)fmax(ceil(p.top_p * (double)total), 1.0); });
    draw_row(lim, false);
  }

  // The list holds every id that min_p keeps (and more): what top_p would
  // keep beyond it falls to min_p anyway.
  __device__ __forceinline__ bool cut_by_min_p(int b) const {
    return p.min_p > 0.0 && b >= (int)fmin(-64.0 * log(p.min_p) + 2.0, (double)(kSampleBins - 2));
  }
};

template <class E>
__global__ __launch_bounds__(kSamplePick) void sample_pick_kernel(SampleArgs A) {
  __shared__ SampleShared s;
  SamplePicker<E> pick(A, s);
  pick.pick();
}

}  // namespace kd
