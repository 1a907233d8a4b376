// kd_sample.hpp -- one token id per row of logits z [R, V], from a uniform
// number given per row.
//
// Per row, with temperature T, m the largest logit and w_v = exp((z_v - m)/T):
// the ids are ordered by (z descending, id ascending); the first top_k stay;
// of these the shortest prefix whose mass reaches top_p of theirs; of these
// the ids with w_v >= min_p.  The drawn id is the first, in id order, whose
// inclusive mass exceeds u times the kept mass.
//
// Borders between ids are decided in 64 bits: w is a double from a polynomial
// (relative error about 1e-14), and masses that ids are picked by are sums of
// 64-bit integers, W_v = rint(w_v 2^s) with s = 62 - ceil(log2 V), at most 51:
// integer sums do not depend on their order, so LDS atomics keep the result
// the same from call to call.  An id more than about 32 T below the largest
// logit (w < 1.3e-14) may count as no mass.  NaN and -inf logits have no mass; a +inf
// logit is the largest and shares the mass with its equals only.
//
// Bound by HBM: R V e bytes, read once by sample_scan_kernel with all of the
// chip (a block per row and 16384 ids): the largest logit of every 64 ids,
// and what the row's filters need: nothing (top_k), the segment's mass (no
// filter), or a histogram of its mass over bins of T/64 (top_p, min_p).  The
// bins lie on a grid of absolute logits, so that no block has to know the
// row's largest logit; a bin's mass is kept relative to its middle, where exp
// needs five terms only.
//
// sample_pick_kernel (a block per row) then
//  - finds from the group maxima (top_k) or from the joined histogram how far
//    below the largest logit kept ids can lie;
//  - when few ids lie that high, reads back only their 64-id groups and ranks
//    them (up to 256 by counting; of a top_k, up to 4096 by sorting);
//  - otherwise (a flat row) reads the row once more for the ids of the border
//    bin alone: the bins above it are kept whole, and the segments' kept
//    masses come from their histograms, so only one segment is looked into.
// Rows that neither suits (more than 4096 ids in the border bin, equal logits
// mostly; top_k past the list; temperatures that put the grid beyond 2^22
// bins) stream the row several times.
#pragma once

#include <type_traits>

#include "kd_layout.hpp"
#include "kd_order.hpp"
#include "kd_rows.hpp"

namespace kd {

constexpr int kSamplePick = 1024;     // threads per row
constexpr int kSampleScan = 512;      // threads per segment
constexpr int kSampleRank = 256;      // longest list that is ranked by counting
constexpr int kSampleSub = 256;       // parts of the border's bins
constexpr float kSampleGrid = 4194304.f;   // largest |logit| in bins that the grid takes

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
  int groups, segs;
  float* gmax;                        // [R][groups] largest logit of a group
  float* smax;                        // [R][segs] of a segment
  double* smass;                      // [R][segs] its mass relative to smax
  int* hlen;                          // [R][segs] bins of its histogram
  uint64_t* hist;                     // [R][segs][kSampleBins], bin 0 that of smax; NULL: V fits the list
  int32_t* token;
  float* logprob;                     // or NULL
};

// A row's parameters: values of a row array outside their range mean "off"
// (top_k < 1 or >= V; top_p >= 1 or NaN; min_p <= 0 or NaN) or the strictest
// setting (temperature <= 0 or NaN: the largest logit; top_p <= 0: the first
// id; min_p > 1: w = 1 only).
struct SampleRow {
  double c64;        // 64 / T: logits in bins
  double step;       // T / 64: a bin in logits
  float cb;          // c64, rounded: bins off the grid, parts of bins
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
  p.c64 = 64.0 / t;
  p.step = t * (1.0 / 64.0);
  p.cb = (float)p.c64;
  return p;
}
// What the scan leaves per segment of a row.
enum SampleScanMode { kScanMax = 0, kScanMass = 1, kScanHist = 2 };
__device__ __forceinline__ int sample_scan_mode(const SampleArgs& A, const SampleRow& p) {
  if (p.greedy || p.top_k > 0) return kScanMax;
  if (p.top_p == 1.0 && p.min_p == 0.0) return kScanMass;
  return kScanHist;
}

// A logit as the operator sees it: NaN as -inf, -0 as +0.
__device__ __forceinline__ float sample_logit(float x) { return fmaxf(x + 0.f, -INFINITY); }

// exp(y / 64) for y <= 1 (0 below -64 * 64 ln 2, and for NaN): 2^k times 2^f,
// |f| <= 1/2, by the Taylor series of exp in f ln 2 up to degree 12 (remainder
// 0.3466^13 / 13! < 2e-16).
__device__ __forceinline__ double exp_bins(double y) {
  constexpr double c[13] = {1.0, 1.0, 1.0 / 2.0, 1.0 / 6.0, 1.0 / 24.0, 1.0 / 120.0, 1.0 / 720.0, 1.0 / 5040.0,
                            1.0 / 40320.0, 1.0 / 362880.0, 1.0 / 3628800.0, 1.0 / 39916800.0, 1.0 / 479001600.0};
  const double z0 = y * (1.4426950408889634 / 64.0);
  const double z = z0 > -64.0 ? z0 : -64.0;        // also NaN (inf - inf, inf * 0)
  const double k = rint(z);
  const double f = (z - k) * 0.6931471805599453;
  double p = c[12];
#pragma unroll
  for (int i = 11; i >= 0; --i) {
    double ci = c[i];
    if (i > 2) asm("" : "+s"(ci));                 // a scalar operand, not a vector register (1 and 1/2 are inline)
    p = fma(p, f, ci);
  }
  // times 2^k, k in [-64, 0], p in [0.7, 1.42]: the exponent field directly
  const double w = __longlong_as_double(__double_as_longlong(p) + (long long)(int)k * (1ll << 52));
  return z0 > -64.0 ? w : 0.0;
}
// exp((l - m) c64 / 64), l <= m.
__device__ __forceinline__ double sample_weight(float l, float m, double c64) {
  return l == m ? 1.0 : exp_bins(((double)l - (double)m) * c64);
}
// The grid of bins: a logit l is in bin rint(l c64), counted from its row's or
// segment's largest.  Added to 1.5 * 2^52 in one step, l c64 is rounded once,
// to the integer in the sum's low bits, so bins are in the logits' order and
// the same wherever they are formed.  Off for largest logits beyond `most`
// bins, infinities, and temperatures so extreme that a bin's logits leave
// fp32's range.
struct SampleGrid {
  static constexpr double kInt = 6755399441055744.0;
  double c64;
  bool on;
  int top;           // bin of the largest logit
  __device__ __forceinline__ SampleGrid(float m, const SampleRow& p, double most) : c64(p.c64) {
    on = p.step > 0x1p-60 && p.step < 0x1p+60 && fabs((double)m * c64) < most;
    top = on ? at(m) : 0;
  }
  __device__ __forceinline__ int at(float l) const { return (int)__double_as_longlong(fma((double)l, c64, kInt)); }
  // The least logit of the bins 0 .. j below the largest one's: the border
  // between two bins (b - 1/2) / c64, rounded to fp32, or its neighbour.
  __device__ __forceinline__ float least(int j, double step) const {
    const int b = top - j;
    const float l = (float)(((double)b - 0.5) * step);        // not 0
    const int up = l > 0.f ? 1 : -1;
    const float below = __int_as_float(__float_as_int(l) - up), above = __int_as_float(__float_as_int(l) + up);
    return at(below) >= b ? below : (at(l) >= b ? l : above);
  }
};
// exp(y / 64) for |y| <= 1/2 (a logit against its bin's middle): degree 5 in
// y / 64, remainder 0.0078^6 / 6! < 4e-16.  The coefficients are held in
// scalar registers, so that a step of the polynomial is one instruction.
struct BinWeight {
  double c[5];
  __device__ __forceinline__ BinWeight() {
    constexpr double h = 1.0 / 64.0;
    c[0] = h;
    c[1] = h * h / 2.0;
    c[2] = h * h * h / 6.0;
    c[3] = h * h * h * h / 24.0;
    c[4] = h * h * h * h * h / 120.0;
#pragma unroll
    for (int i = 0; i < 5; ++i) asm("" : "+s"(c[i]));
  }
  __device__ __forceinline__ double operator()(double y) const {
    double p = fma(c[4], y, c[3]);
    p = fma(p, y, c[2]);
    p = fma(p, y, c[1]);
    p = fma(p, y, c[0]);
    return fma(p, y, 1.0);
  }
};
// Units of the masses, 2^s.
__device__ __forceinline__ double sample_scale(int V) {
  const int bits = 62 - (32 - __clz(max(V - 1, 1)));
  return (double)(1ull << min(bits, 51));
}
// rint(w * scale) for products below 2^52: added to 2^52 the integer is the
// low bits of the sum.
__device__ __forceinline__ uint64_t sample_units(double w, double scale) {
  return (uint64_t)__double_as_longlong(fma(w, scale, 4503599627370496.0)) - 0x4330000000000000ull;
}

// 16 bytes of consecutive logits of a row (-inf past its end); RAW: NaN stays.
template <class E> struct SampleVec;
template <> struct SampleVec<Bf16> { static constexpr int N = 8; };
template <> struct SampleVec<F32> { static constexpr int N = 4; };
template <class E, bool RAW = false>
__device__ __forceinline__ void sample_load(const typename E::T* row, int v, int V, float* x) {
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
  for (int i = 0; i < N; ++i) x[i] = RAW ? x[i] + 0.f : sample_logit(x[i]);
}

// The larger of two numbers that are not signalling NaN; of a number and a
// NaN the number.  (fmaxf quiets its arguments first: two instructions more.)
__device__ __forceinline__ float quiet_max(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
// Each of g's values becomes the maximum over the 16 (eight values) or 8 lanes
// (four) that share a group, by maxima whose second operand is another lane's:
// those that a DPP reads were written three instructions before at least (two
// are the least), the first ones by the wait.
__device__ __forceinline__ void group_max(float (&g)[8]) {
#define KD_STEP(c)                                                                                                   \
  "v_max_f32_dpp %0, %0, %0 " c "\n\tv_max_f32_dpp %1, %1, %1 " c "\n\tv_max_f32_dpp %2, %2, %2 " c                  \
  "\n\tv_max_f32_dpp %3, %3, %3 " c "\n\tv_max_f32_dpp %4, %4, %4 " c "\n\tv_max_f32_dpp %5, %5, %5 " c             \
  "\n\tv_max_f32_dpp %6, %6, %6 " c "\n\tv_max_f32_dpp %7, %7, %7 " c "\n\t"
  asm("s_nop 4\n\t" KD_STEP("quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf")
      KD_STEP("quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf") KD_STEP("row_half_mirror row_mask:0xf bank_mask:0xf")
      KD_STEP("row_mirror row_mask:0xf bank_mask:0xf")
      : "+v"(g[0]), "+v"(g[1]), "+v"(g[2]), "+v"(g[3]), "+v"(g[4]), "+v"(g[5]), "+v"(g[6]), "+v"(g[7]));
#undef KD_STEP
}
__device__ __forceinline__ void group_max(float (&g)[4]) {
#define KD_STEP(c)                                                                                                   \
  "v_max_f32_dpp %0, %0, %0 " c "\n\tv_max_f32_dpp %1, %1, %1 " c "\n\tv_max_f32_dpp %2, %2, %2 " c                  \
  "\n\tv_max_f32_dpp %3, %3, %3 " c "\n\t"
  asm("s_nop 4\n\t" KD_STEP("quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf")
      KD_STEP("quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf") KD_STEP("row_half_mirror row_mask:0xf bank_mask:0xf")
      : "+v"(g[0]), "+v"(g[1]), "+v"(g[2]), "+v"(g[3]));
#undef KD_STEP
}

// A block per row and segment; 32 ids per thread, held in registers, 64
// registers in all (full occupancy).  256 fp32 rows of 201088 with top_p from
// HBM take 60 us (3.4 TB/s), 50 with neither masses nor histogram: reading
// bounds it, a block's phases (read, largest logit, histogram, write) one
// after the other keep it below a copy's rate.  Bins by fp32 products and
// floors, with a polynomial of one more degree about the bin's edge, took 62.5.
template <class E>
__global__ __launch_bounds__(kSampleScan) void sample_scan_kernel(SampleArgs A) {
  constexpr int N = SampleVec<E>::N, L = kSampleSeg / (N * kSampleScan);
  __shared__ float s_max[kSampleScan / 64];
  __shared__ double s_sum[kSampleScan / 64];
  __shared__ int s_len;
  __shared__ unsigned long long s_hist[kSampleBins];
  const int r = blockIdx.x / A.segs, seg = blockIdx.x - r * A.segs;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const typename E::T* row = (const typename E::T*)A.z + (int64_t)r * A.ldz;
  float x[L][N];
#pragma unroll
  for (int j = 0; j < L; ++j) sample_load<E, true>(row, seg * kSampleSeg + (j * kSampleScan + tid) * N, A.V, x[j]);
  const SampleRow p = sample_row(A, r);
  const int mode = sample_scan_mode(A, p);
  static_assert(kSampleGroup / N == (L == 8 ? 16 : 8), "lanes of a group");
  float m = -INFINITY, g[L];
#pragma unroll
  for (int j = 0; j < L; ++j) {
    g[j] = -INFINITY;                              // (stays where all are NaN)
#pragma unroll
    for (int i = 0; i < N; ++i) g[j] = quiet_max(g[j], x[j][i]);
  }
  group_max(g);
#pragma unroll
  for (int j = 0; j < L; ++j) {
    const int gi = seg * (kSampleSeg / kSampleGroup) + (j * kSampleScan + tid) * N / kSampleGroup;
    if (lane % (kSampleGroup / N) == 0 && gi < A.groups) A.gmax[(int64_t)r * A.groups + gi] = g[j];
    m = quiet_max(m, g[j]);
  }
  // (the compiler, which keeps a lane-crossing read two instructions behind its
  // operand's last write, does not see the one in quiet_max)
  asm("s_nop 1" : "+v"(m));
  m = wave_max(m);
  if (lane == 0) s_max[wave] = m;
  if (mode == kScanHist && A.hist)
    for (int i = tid; i < kSampleBins; i += kSampleScan) s_hist[i] = 0;
  if (tid == 0) s_len = 0;
  __syncthreads();
  m = s_max[0];
#pragma unroll
  for (int i = 1; i < kSampleScan / 64; ++i) m = fmaxf(m, s_max[i]);
  const int64_t at = (int64_t)r * A.segs + seg;
  if (tid == 0) A.smax[at] = m;
  // ids below the last bin with mass go to the one after it, and so does NaN
  const SampleGrid grid(m, p, kSampleGrid);
  const float bottom = (float)((double)(grid.top - (kSampleBins - 1)) * p.step);
  // the bin of an id and its weight relative to the bin's middle
  double whole = SampleGrid::kInt;
  asm("" : "+s"(whole));
  auto place = [&](const BinWeight& weight, float l, int& d) {
    const double x = (double)quiet_max(l, bottom), t = fma(x, p.c64, whole);
    d = grid.top - (int)__double_as_longlong(t);
    return weight(fma(x, p.c64, whole - t));
  };
  if (mode == kScanMass) {
    double s = 0.0;
    if (grid.on) {                                 // (uniform)
      // exp((l - m) / T) as the factor of the logit's bin, from a table, and
      // the five terms of its place in the bin
      double* factor = (double*)s_hist;
      for (int i = tid; i < kSampleBins; i += kSampleScan)
        factor[i] = i < kSampleBins - 1 ? exp_bins(fma((double)m, -p.c64, (double)(grid.top - i))) : 0.0;
      __syncthreads();
      const BinWeight weight;
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int q = 0; q < N; q += 2) {
          // two ids at a time: their polynomials interleave, and the kernel
          // stays within 64 registers (eight waves per SIMD)
          double w[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            int d;
            w[i] = place(weight, x[j][q + i], d);
            w[i] *= factor[d];
          }
          s += w[0] + w[1];
          asm volatile("" : "+v"(s));
        }
    } else if (m > -INFINITY) {
      // (read again: few rows come here)
#pragma unroll 1
      for (int i = tid; i < kSampleSeg && seg * kSampleSeg + i < A.V; i += kSampleScan)
        s += sample_weight(sample_logit(load_elem<E>(row + seg * kSampleSeg + i)), m, p.c64);
    }
    s = wave_sum(s);
    if (lane == 0) s_sum[wave] = s;
    __syncthreads();
    if (tid == 0) {
      s = 0.0;
      for (int i = 0; i < kSampleScan / 64; ++i) s += s_sum[i];
      A.smass[at] = s;
    }
  } else if (mode == kScanHist && A.hist) {
    int last = -1;
    if (grid.on) {
      const double scale = sample_scale(A.V);
      const BinWeight weight;
#pragma unroll
      for (int j = 0; j < L; ++j)
#pragma unroll
        for (int q = 0; q < N; q += 4) {
          // four ids at a time: their polynomials interleave
          int d[4];
          uint64_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = sample_units(place(weight, x[j][q + i], d[i]), scale);
            asm volatile("" : "+v"(w[i]), "+v"(d[i]));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (d[i] < kSampleBins - 1) {
              atomicAdd(&s_hist[d[i]], (unsigned long long)w[i]);
              last = max(last, d[i]);
            }
        }
    }
    if (last >= 0) atomicMax(&s_len, last + 1);
    __syncthreads();
    const int len = s_len;
    if (tid == 0) A.hlen[at] = len;
    uint64_t* out = A.hist + at * kSampleBins;
    for (int i = tid; i < len; i += kSampleScan) out[i] = s_hist[i];
  }
}

// ---------------------------------------------------------------------------
// One block per row.
// ---------------------------------------------------------------------------
struct SampleShared {
  uint64_t key[kSampleList];       // candidates: cand_key(z, id)
  uint64_t aux[kSampleList];       // group lists; masses; keys by id; bin factors
  uint64_t bins[kSampleBins];      // histograms; kept masses of the segments
  uint64_t red[kSamplePick / 64];
  uint64_t sub[kSampleSub];        // mass of the border's sub-bins
  int n, n2, pos;
  uint64_t a;
};

// The sixteen waves' values, prefix-summed by every wave for itself: lane i
// of its first sixteen holds the sum of waves 0 .. i.
template <class T>
__device__ __forceinline__ T waves_scan(SampleShared& s, T v) {
  static_assert(kSamplePick == 1024, "sixteen waves");
  if ((threadIdx.x & 63) == 63) s.red[threadIdx.x >> 6] = __builtin_bit_cast(uint64_t, v);
  __syncthreads();
  T t = __builtin_bit_cast(T, s.red[threadIdx.x & 15]);
  t += dpp<0x111>(t);
  t += dpp<0x112>(t);
  t += dpp<0x114>(t);
  t += dpp<0x118>(t);
  __syncthreads();
  return t;
}
// Inclusive prefix sum over the block's threads; their total in `total`.
template <class T>
__device__ __forceinline__ T block_scan(SampleShared& s, T v, T& total) {
  v = wave_incl_scan(v);
  const T t = waves_scan(s, v);
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  total = read_lane(t, 15);
  return w ? read_lane(t, (w - 1) & 15) + v : v;
}
template <class T>
__device__ __forceinline__ T block_total(SampleShared& s, T v) {
  return read_lane(waves_scan(s, wave_sum(v)), 15);
}

// The first of n positions whose inclusive prefix reaches `target` > 0
// (-1: none), and the prefix before it; value(i) is called once per position.
template <class T, class F>
__device__ __forceinline__ int block_find(SampleShared& s, int n, T target, F value, T& before) {
  T base = 0;
  for (int i0 = 0; i0 < n; i0 += kSamplePick) {
    const int i = i0 + (int)threadIdx.x;
    const T v = i < n ? value(i) : 0;
    T total;
    const T incl = base + block_scan(s, v, total);
    if (base + total >= target) {                  // uniform
      if constexpr (std::is_integral<T>::value) {
        if (incl >= target && incl - v < target) { // exactly one thread
          s.pos = i;
          s.a = incl - v;
        }
      } else {
        // rounding may leave several threads, or a position past n, that
        // look like the border: the lowest is taken
        if (threadIdx.x == 0) s.pos = 0x7fffffff;
        __syncthreads();
        if (incl >= target) atomicMin(&s.pos, i);
        __syncthreads();
        if (i == min(s.pos, n - 1)) s.a = __builtin_bit_cast(uint64_t, incl - v);
      }
      __syncthreads();
      const int pos = min(s.pos, n - 1);
      before = __builtin_bit_cast(T, s.a);
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

// Sort key[0, n) descending (padding to a power of two with zeros).
__device__ __forceinline__ void sort_keys(uint64_t* key, int n) {
  const int m = pow2_at_least(n);
  for (int i = n + (int)threadIdx.x; i < m; i += kSamplePick) key[i] = 0;
  __syncthreads();
  bitonic_desc(key, m);
}

__device__ __forceinline__ SampleShared& sample_shared() {
  __shared__ SampleShared s;
  return s;
}
template <class E>
__device__ __attribute__((noinline)) void sample_stream_row(SampleArgs A, float m);

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
  float m;                     // the largest logit
  SampleGrid grid;             // on: bins are the scan's
  double scale;

  __device__ explicit SamplePicker(const SampleArgs& a)
      : A(a), s(sample_shared()), r(blockIdx.x), p(sample_row(a, blockIdx.x)), row((const T*)a.z + (int64_t)blockIdx.x * a.ldz),
        gmax(a.gmax + (int64_t)blockIdx.x * a.groups), grid(INFINITY, p, 0.0), scale(sample_scale(a.V)) {}

  // Bin of a logit below the largest: non-decreasing as l falls.  The last
  // bin has no mass.
  __device__ __forceinline__ int bin(float l) const {
    if (l == m) return 0;
    const float x = (m - l) * p.cb;
    const float y = fminf(x, (float)(kSampleBins - 1));      // NaN (inf * 0): the last bin
    // (a logit two bins past the last one is not formed on the grid, where it could leave 32 bits)
    return grid.on && x < (float)(kSampleBins + 1) ? min(grid.top - grid.at(l), kSampleBins - 1) : (int)y;
  }
  __device__ __forceinline__ uint64_t mass(float l) const {
    return sample_units(sample_weight(l, m, p.c64), scale);
  }
  // The mass if the id passes min_p, else 0.
  __device__ __forceinline__ uint64_t kept_mass(float l) const {
    const double w = sample_weight(l, m, p.c64);
    return w >= p.min_p ? sample_units(w, scale) : 0;
  }
  __device__ __forceinline__ bool passes_min_p(float l) const {
    return p.min_p == 0.0 || sample_weight(l, m, p.c64) >= p.min_p;
  }
  // The smallest inclusive prefix that exceeds u * total (1 .. total).
  __device__ __forceinline__ uint64_t draw_target(uint64_t total) const {
    const double u = A.u_is_f64 ? ((const double*)A.u)[r] : (double)((const float*)A.u)[r];
    const double x = floor(u * (double)total);
    if (!(x > 0.0)) return 1;                      // also a NaN
    return x >= (double)total ? total : min((uint64_t)x + 1, total);
  }
  // One thread writes the result.
  __device__ __forceinline__ void emit(int id, float l, uint64_t total) const {
    A.token[r] = id;
    // ln w of the drawn id minus the ln of the kept mass
    if (A.logprob)
      A.logprob[r] = (float)((l == m ? 0.0 : ((double)l - (double)m) * p.c64 * (1.0 / 64.0)) - log((double)total / scale));
  }

  // Calls f(group, its largest logit) for every group, each thread a strided
  // share, four loads in flight.
  template <class F>
  __device__ __forceinline__ void for_groups(F f) const {
    for (int i = threadIdx.x; i < A.groups; i += 4 * kSamplePick) {
      float g[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = i + j * kSamplePick < A.groups ? gmax[i + j * kSamplePick] : -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (g[j] > -INFINITY) f(i + j * kSamplePick, g[j]);
    }
  }

  // Lowest id of the largest logit.
  __device__ __forceinline__ void pick_greedy() {
    if (threadIdx.x == 0) s.pos = A.groups;
    __syncthreads();
    for_groups([&](int i, float g) {
      if (g == m) atomicMin(&s.pos, i);
    });
    __syncthreads();
    if (threadIdx.x < 64) {
      const int v = s.pos * kSampleGroup + (int)threadIdx.x;
      const bool hit = v < A.V && sample_logit(load_elem<E>(row + v)) == m;
      const unsigned long long b = __ballot(hit);
      if (threadIdx.x == 0) {
        A.token[r] = s.pos * kSampleGroup + (int)__builtin_ctzll(b);
        if (A.logprob) A.logprob[r] = 0.f;
      }
    }
  }

  // Bin that `want` groups have their maxima in or above (the last one with
  // mass if there are fewer).
  __device__ __forceinline__ int group_bin(int want) {
    int* cnt = (int*)s.bins;
    for (int i = threadIdx.x; i < kSampleBins; i += kSamplePick) cnt[i] = 0;
    __syncthreads();
    for_groups([&](int, float g) { atomicAdd(&cnt[bin(g)], 1); });
    __syncthreads();
    uint64_t before;
    // two bins per thread: one prefix sum covers them all
    const int b = block_find(
        s, kSampleBins / 2, (uint64_t)want,
        [&](int i) -> uint64_t { return cnt[2 * i] + (2 * i + 1 < kSampleBins - 1 ? cnt[2 * i + 1] : 0); }, before);
    if (b < 0) return kSampleBins - 2;
    return before + cnt[2 * b] >= (uint64_t)want ? 2 * b : 2 * b + 1;
  }

  // All ids in bins <= b into s.key (unordered), if their groups are at most
  // `most`; their number, or one past kSampleList if they do not fit.  The
  // groups that hold them are left as bits in group_bits().
  __device__ __forceinline__ uint64_t* group_bits() const { return s.aux; }          // one per group ..
  __device__ __forceinline__ bool has_bits() const { return A.groups <= 64 * (kSampleList / 2); }   // .. if they fit half of aux
  __device__ __forceinline__ int gather(int b, int most) {
    int* list = (int*)(s.aux + kSampleList / 2);   // groups to read: kSampleList places
    if (threadIdx.x == 0) s.n = s.n2 = 0;
    __syncthreads();
    const bool bits = has_bits();
    for (int i = threadIdx.x; i - (int)threadIdx.x < A.groups; i += 4 * kSamplePick) {   // whole waves
      float g[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = i + j * kSamplePick < A.groups ? gmax[i + j * kSamplePick] : -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int gi = i + j * kSamplePick;
        const bool in = g[j] > -INFINITY && bin(g[j]) <= b;
        const unsigned long long w = __ballot(in);
        if (bits && (gi & 63) == 0 && gi < A.groups) group_bits()[gi / 64] = w;
        if (w) {
          int at = 0;                              // one count per wave
          if ((threadIdx.x & 63) == 0) at = atomicAdd(&s.n2, (int)__popcll(w));
          at = __builtin_amdgcn_readfirstlane(at) +
               (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(w >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)w, 0));
          if (in && at < kSampleList) list[at] = gi;
        }
      }
    }
    __syncthreads();
    const int ng = s.n2;
    if (ng > most) return kSampleList + 1;
    const int lane = threadIdx.x & 63;
    constexpr int D = 8;                           // groups per wave in flight
    constexpr int W = kSamplePick / 64;
    for (int g0 = threadIdx.x >> 6; g0 < ng; g0 += D * W) {
      float x[D];
      int v[D];
#pragma unroll
      for (int j = 0; j < D; ++j) {
        v[j] = g0 + j * W < ng ? list[g0 + j * W] * kSampleGroup + lane : A.V;
        x[j] = v[j] < A.V ? sample_logit(load_elem<E>(row + v[j])) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < D; ++j)
        if (v[j] < A.V && bin(x[j]) <= b) {
          const int at = atomicAdd(&s.n, 1);
          if (at < kSampleList) s.key[at] = cand_key(x[j], (uint32_t)v[j]);
        }
    }
    __syncthreads();
    const int n = s.n;
    __syncthreads();                               // the caller may clear it
    return n;
  }

  // Draw from the n <= kSampleRank ids of s.key (any order), by counting: per
  // id, how many stand before it and with what mass.  All prefixes are sums
  // over the list, split over the block's threads and joined with integer
  // atomics.  row_mass: the mass that top_p is a share of when top_k is off.
  __device__ __forceinline__ void draw_few(int n, double row_mass) {
    uint64_t* wt = s.aux;                          // masses
    uint64_t* pre = s.aux + kSampleRank;           // mass before, by rank; then inclusive mass, by id
    int* rank = (int*)(s.aux + 2 * kSampleRank);
    const int tid = threadIdx.x, i = tid & (kSampleRank - 1), q = tid / kSampleRank;
    constexpr int Q = kSamplePick / kSampleRank;
    uint64_t k = 0, w = 0;
    if (i < n) {
      k = s.key[i];
      w = mass(key_logit(k));
    }
    if (q == 0) {
      wt[i] = w;
      pre[i] = 0;
      rank[i] = 0;
    }
    __syncthreads();
    if (i < n) {
      int c = 0;
      uint64_t a = 0;
#pragma unroll 4
      for (int j = q; j < n; j += Q)
        if (s.key[j] > k) {
          ++c;
          a += wt[j];
        }
      atomicAdd(&rank[i], c);
      atomicAdd((unsigned long long*)&pre[i], (unsigned long long)a);
    }
    __syncthreads();
    bool keep = i < n && (p.top_k == 0 || rank[i] < p.top_k);
    if (p.top_p < 1.0) {
      const double all = p.top_k > 0 ? (double)block_total(s, q == 0 && keep ? w : (uint64_t)0) : row_mass;
      keep = keep && (rank[i] == 0 || (double)pre[i] < p.top_p * all);
    }
    keep = keep && w > 0 && passes_min_p(key_logit(k));
    __syncthreads();
    if (q == 0) {
      wt[i] = keep ? w : 0;
      pre[i] = 0;
    }
    const uint64_t total = block_total(s, q == 0 && keep ? w : (uint64_t)0);   // its barriers order the writes
    if (keep) {
      uint64_t a = 0;
#pragma unroll 4
      for (int j = q; j < n; j += Q)
        if ((uint32_t)s.key[j] >= (uint32_t)k) a += wt[j];       // ids <= this one
      atomicAdd((unsigned long long*)&pre[i], (unsigned long long)a);
    }
    __syncthreads();
    const uint64_t want = draw_target(total);
    if (q == 0 && keep && pre[i] >= want && pre[i] - w < want) emit(key_id(k), key_logit(k), total);
  }

  // Draw from the first n entries of s.key that pass min_p: sorted by id.
  __device__ __forceinline__ void draw_list(int n) {
    // aux: (~id, position) keys, largest first = lowest id first; entries
    // that are not kept are zero and sort last
    for (int i = threadIdx.x; i < n; i += kSamplePick)
      s.aux[i] = passes_min_p(key_logit(s.key[i])) ? (((uint64_t)(uint32_t)s.key[i]) << 32) | (uint32_t)i : 0;
    __syncthreads();
    sort_keys(s.aux, n);
    auto value = [&](int i) -> uint64_t {
      const uint64_t a = s.aux[i];
      return a ? mass(key_logit(s.key[(uint32_t)a])) : 0;
    };
    uint64_t part = 0, before;
    for (int i = threadIdx.x; i < n; i += kSamplePick) part += value(i);
    const uint64_t total = block_total(s, part);
    const int at = block_find(s, n, draw_target(total), value, before);
    const uint64_t k = s.key[(uint32_t)s.aux[max(at, 0)]];
    if (threadIdx.x == 0) emit(key_id(k), key_logit(k), total);
  }

  // Draw from a list that holds every id in bins <= some bin, and so every
  // kept one.
  __device__ __forceinline__ void pick_list(int n, double row_mass) {
    if (n <= kSampleRank) return draw_few(n, row_mass);
    int n1 = n;
    if (p.top_k > 0 || p.top_p < 1.0) {
      sort_keys(s.key, n);
      if (p.top_k > 0) n1 = min(n, p.top_k);
    }
    if (p.top_p < 1.0) {
      auto value = [&](int i) { return mass(key_logit(s.key[i])); };
      double all = row_mass;
      if (p.top_k > 0) {
        uint64_t part = 0;
        for (int i = threadIdx.x; i < n1; i += kSamplePick) part += value(i);
        all = (double)block_total(s, part);
      }
      uint64_t before;
      const int at = block_find(s, n1, (uint64_t)fmax(ceil(p.top_p * all), 1.0), value, before);
      if (at >= 0) n1 = at + 1;
    }
    draw_list(n1);
  }

  // ---- flat rows, from the scan's histograms -------------------------------
  // Mass of bin j of the row relative to the largest logit: its entries are
  // kept relative to the bin's middle, top - j on the grid.
  __device__ __forceinline__ double bin_factor(int j) const {
    return exp_bins(fma((double)m, -p.c64, (double)(grid.top - j)));
  }
  __device__ __forceinline__ int seg_offset(int sg) const {
    // bins between the row's largest logit and the segment's
    return bin(A.smax[(int64_t)r * A.segs + sg]);  // -inf: the last one
  }

  // The kept set: every id with l >= edge (NaN: none) and, below it, those that
  // are not after the id `last` with the logit `least` in descending order.
  struct Kept {
    float edge, least;
    int last;
  };
  // cand_key >= lim (0: all above -inf; ~0: none)
  __device__ __forceinline__ static Kept kept_from(float edge, uint64_t lim) {
    if (lim == 0) return Kept{edge, -INFINITY, -1};
    return lim == ~0ull ? Kept{edge, INFINITY, -1} : Kept{edge, key_logit(lim), key_id(lim)};
  }
  __device__ __forceinline__ bool is_kept(const Kept& k, int v, float l) const {
    return l >= k.edge || l > k.least || (l == k.least && v <= k.last);
  }

  // Draw, given the segments' kept masses in s.bins.  A segment whose mass
  // is less than the rounding of its ids' (none of them has a unit) is left
  // out and the draw repeated; the largest logit's segment always stays.
  __device__ __forceinline__ void draw_segment(const Kept& k) {
    while (!try_segment(k)) {}
  }
  __device__ __forceinline__ bool try_segment(const Kept& k) {
    uint64_t part = 0, before = 0;
    for (int i = threadIdx.x; i < A.segs; i += kSamplePick) part += s.bins[i];
    const uint64_t total = block_total(s, part);
    const uint64_t want = draw_target(total);
    const int sg = max(block_find(s, A.segs, want, [&](int i) { return s.bins[i]; }, before), 0);
    // 16 consecutive ids per thread
    constexpr int C = kSampleSeg / kSamplePick;
    const int v0 = sg * kSampleSeg + (int)threadIdx.x * C;
    float x[C];
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < C / N; ++j) sample_load<E>(row, v0 + j * N, A.V, x + j * N);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      sum += is_kept(k, v0 + i, x[i]) ? kept_mass(x[i]) : 0;
      if (i & 1) asm volatile("" : "+v"(sum));     // two at a time: few registers
    }
    uint64_t all;
    uint64_t run = block_scan(s, sum, all) - sum;
    if (all == 0) {
      if (threadIdx.x == 0) s.bins[sg] = 0;
      __syncthreads();
      return false;
    }
    // (a segment's mass taken from its histogram may differ from this sum in
    // the last units: the target is held inside it)
    const uint64_t aim = min(want > before ? want - before : (uint64_t)1, all);
    if (run < aim && run + sum >= aim) {           // one thread; its ids to a wave
      s.pos = v0;
      s.a = run;
    }
    __syncthreads();
    if (threadIdx.x < 64) {
      const int v = s.pos + (int)threadIdx.x;
      const float l = (int)threadIdx.x < C && v < A.V ? sample_logit(load_elem<E>(row + v)) : -INFINITY;
      const uint64_t w = is_kept(k, v, l) ? kept_mass(l) : 0;
      const uint64_t incl = s.a + wave_incl_scan(w);
      if (w && incl >= aim && incl - w < aim) emit(v, l, total);
    }
    return true;
  }

  // top_p and min_p without top_k: the row's histogram into s.bins; returns
  // the mass of the row, the bins lo .. hi that the kept set ends in, and about
  // how many ids lie in the bins up to hi (each has a mass within a hundredth
  // of one unit of its bin's).
  __device__ __forceinline__ double join_hist(int& lo, int& hi, double& ids) {
    const int64_t at0 = (int64_t)r * A.segs;
    double* bm = (double*)s.bins;
    // per segment: where its histogram starts among the row's bins, its length
    int2* seg = (int2*)s.aux;
    for (int sg = threadIdx.x; sg < A.segs; sg += kSamplePick) seg[sg] = make_int2(seg_offset(sg), A.hlen[at0 + sg]);
    __syncthreads();
    static_assert(kSampleBins == 2 * kSamplePick, "two bins per thread");
    const int j0 = threadIdx.x, j1 = j0 + kSamplePick;
    uint64_t a0 = 0, a1 = 0;
#pragma unroll 8
    for (int sg = 0; sg < A.segs; ++sg) {
      const int2 at = seg[sg];
      const uint64_t* h = A.hist + (at0 + sg) * kSampleBins - at.x;
      a0 += j0 >= at.x && j0 - at.x < at.y ? h[j0] : 0;
      a1 += j1 >= at.x && j1 - at.x < at.y ? h[j1] : 0;
    }
    bm[j0] = a0 ? (double)a0 * bin_factor(j0) : 0.0;
    bm[j1] = a1 && j1 < kSampleBins - 1 ? (double)a1 * bin_factor(j1) : 0.0;
    const double part = bm[j0] + bm[j1];
    const double all = block_total(s, part);       // (orders the writes)
    const double need = p.top_p * all;
    lo = kSampleBins - 1;
    hi = kSampleBins - 2;
    if (p.min_p > 0.0) {
      // w >= min_p: at most x bins below the largest logit; a bin's ids lie
      // within one bin of its number, and one more for rounding
      const double x = fmin(-64.0 * log(p.min_p), (double)(2 * kSampleBins));
      lo = min(max((int)x - 1, 0), lo);
      hi = min((int)x + 2, hi);
    }
    if (p.top_p < 1.0) {
      double before;
      const int b = block_find(s, kSampleBins / 2, need, [&](int i) { return bm[2 * i] + bm[2 * i + 1]; }, before);
      const int jb = b < 0 ? kSampleBins - 2 : (before + bm[2 * b] >= need ? 2 * b : 2 * b + 1);
      lo = min(lo, jb);
      hi = min(hi, jb);
    }
    ids = block_total(s, (j0 <= hi ? (double)a0 : 0.0) + (j1 <= hi ? (double)a1 : 0.0)) / scale;
    return all;
  }

  // The kept set of a flat row, given its histogram in s.bins, and the
  // segments' kept masses in its place.  False: the border holds too many ids.
  __device__ __forceinline__ bool cut_hist(double all, int lo, int hi, Kept& k) {
    const int64_t at0 = (int64_t)r * A.segs;
    const double* bm = (const double*)s.bins;
    const double need = p.top_p * all;
    // the border's ids, bins lo .. hi: lb <= l < ub
    if (threadIdx.x == 0) s.n = s.n2 = 0;
    for (int i = threadIdx.x; i < kSampleSub; i += kSamplePick) s.sub[i] = 0;
    double part = 0.0;
    for (int j = threadIdx.x; j < lo; j += kSamplePick) part += bm[j];
    const double above = block_total(s, part);     // (orders the writes above)
    const float lb = grid.least(hi, p.step), ub = lo > 0 ? grid.least(lo - 1, p.step) : INFINITY;
    // parts of the border, in the logits' order
    const float per = (float)kSampleSub / (float)(hi - lo + 1), first = (float)(grid.top - lo) + 0.5f;
    auto part_of = [&](float l) { return min(max((int)((first - l * p.cb) * per), 0), kSampleSub - 1); };
    // 32 ids per thread and step: a bit each for those in the border, whose
    // ids then go to the list (hardly any lane has more than two)
    constexpr int D = 32 / N;
    const bool bits = has_bits();
    int* ids = (int*)s.key;
    for (int v = (int)threadIdx.x * N; v < A.V; v += kSamplePick * 32) {
      // (of groups with an id that high: the others are not read)
      u32x4 u[D];
#pragma unroll
      for (int j = 0; j < D; ++j) {
        const int vj = v + j * kSamplePick * N, g = vj / kSampleGroup;
        u[j] = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};   // NaN of both types: in no bin
        if (vj + N <= A.V && (!bits || (group_bits()[g / 64] >> (g & 63)) & 1)) __builtin_memcpy(&u[j], row + vj, 16);
      }
      uint32_t hits = 0;
#pragma unroll
      for (int j = 0; j < D; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float l;
          if constexpr (N == 8) l = __uint_as_float((i & 1) ? (u[j][i >> 1] & 0xffff0000u) : (u[j][i >> 1] << 16));
          else l = __uint_as_float(u[j][i]);
          hits |= l >= lb && l < ub ? 1u << (j * N + i) : 0u;
        }
      while (hits) {
        const int q = __builtin_ctz(hits);
        hits &= hits - 1;
        const int at = atomicAdd(&s.n, 1);
        if (at < kSampleList) ids[at] = v + (q / N) * (kSamplePick * N) + q % N;
      }
    }
    // the last vector, where it crosses the row's end
    if (threadIdx.x < A.V % N) {
      const int v = A.V - A.V % N + (int)threadIdx.x;
      const float l = load_elem<E>(row + v);
      if (l >= lb && l < ub) {
        const int at = atomicAdd(&s.n, 1);
        if (at < kSampleList) ids[at] = v;
      }
    }
    __syncthreads();
    const int n = s.n;
    __syncthreads();
    if (n > kSampleList) return false;
    // ids to keys, and the mass of each part of the border
    constexpr int P = kSampleList / kSamplePick;
    uint64_t key[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = (int)threadIdx.x + j * kSamplePick;
      key[j] = 0;
      if (i < n) key[j] = cand_key(sample_logit(load_elem<E>(row + ids[i])), (uint32_t)ids[i]);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int i = (int)threadIdx.x + j * kSamplePick;
      if (i >= n) continue;
      s.key[i] = key[j];
      if (p.top_p < 1.0) {
        const float l = key_logit(key[j]);
        atomicAdd((unsigned long long*)&s.sub[part_of(l)], (unsigned long long)mass(l));
      }
    }
    __syncthreads();
    // which of them stay: those that pass min_p and, with top_p, the whole
    // sub-bins above the one where their mass reaches its share, and of that
    // one's ids, sorted, the first
    uint64_t lim = 0;
    if (p.top_p < 1.0) {
      if (need <= above && lo > 0) {
        lim = ~0ull;
      } else {
        const uint64_t want = (uint64_t)fmax(ceil(need - above), 1.0);
        uint64_t before;
        const int sb = block_find(s, kSampleSub, want, [&](int i) { return s.sub[i]; }, before);
        if (sb >= 0) {
          for (int i = threadIdx.x; i < n; i += kSamplePick)
            if (part_of(key_logit(s.key[i])) == sb) s.aux[atomicAdd(&s.n2, 1)] = s.key[i];
          __syncthreads();
          const int ns = s.n2;
          __syncthreads();
          sort_keys(s.aux, ns);
          const int at = block_find(s, ns, want - before, [&](int i) { return mass(key_logit(s.aux[i])); }, before);
          lim = s.aux[at < 0 ? ns - 1 : at];
          __syncthreads();
        }
      }
    }
    k = kept_from(ub, lim);
    // the segments' masses above the border, a wave per segment, then the
    // border's kept ids
    double* fac = (double*)s.aux;
    for (int j = threadIdx.x; j < lo; j += kSamplePick) fac[j] = bin_factor(j);
    __syncthreads();
    for (int sg = threadIdx.x >> 6; sg < A.segs; sg += kSamplePick / 64) {
      const int off = seg_offset(sg), len = min(A.hlen[at0 + sg], lo - off);
      const uint64_t* h = A.hist + (at0 + sg) * kSampleBins;
      double v = 0.0;
#pragma unroll 8
      for (int i = threadIdx.x & 63; i < len; i += 64) v += (double)h[i] * fac[off + i];
      v = wave_sum(v);
      if ((threadIdx.x & 63) == 0) s.bins[sg] = (uint64_t)rint(v);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSamplePick) {
      const uint64_t c = s.key[i];
      const uint64_t w = c >= lim ? kept_mass(key_logit(c)) : 0;
      if (w) atomicAdd((unsigned long long*)&s.bins[key_id(c) / kSampleSeg], (unsigned long long)w);
    }
    __syncthreads();
    return true;
  }

  // ---- rows that are streamed several times --------------------------------
  // Calls f(id, logit) for every id of the row above -inf, each thread a
  // strided share.
  template <class F>
  __device__ __forceinline__ void for_row(F f) {
    constexpr int D = 32 / N;                      // loads in flight
    for (int v = (int)threadIdx.x * N; v < A.V; v += kSamplePick * N * D) {
      float x[D][N];
#pragma unroll
      for (int j = 0; j < D; ++j) sample_load<E>(row, v + j * kSamplePick * N, A.V, x[j]);
#pragma unroll
      for (int j = 0; j < D; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (x[j][i] > -INFINITY) f(v + j * kSamplePick * N + i, x[j][i]);
    }
  }

  // Tighten `lim` (kept: cand_key >= lim) to the shortest prefix, in
  // descending order, of the kept ids with mass whose count (MASS false) or
  // mass reaches a target; target(total) gives it from their total.
  template <bool MASS, class F>
  __device__ __forceinline__ uint64_t cut(uint64_t lim, F target) {
    for (int i = threadIdx.x; i < kSampleBins; i += kSamplePick) s.bins[i] = 0;
    __syncthreads();
    for_row([&](int v, float l) {
      const int b = bin(l);
      if (b < kSampleBins - 1 && cand_key(l, (uint32_t)v) >= lim)
        atomicAdd((unsigned long long*)&s.bins[b], MASS ? (unsigned long long)mass(l) : 1ull);
    });
    __syncthreads();
    uint64_t part = 0;
    for (int i = threadIdx.x; i < kSampleBins; i += kSamplePick) part += s.bins[i];
    const uint64_t want = target(block_total(s, part));
    uint64_t before;
    const int b = block_find(s, kSampleBins - 1, want, [&](int i) { return s.bins[i]; }, before);
    if (b < 0) return lim;                         // the target is not reached: all stay
    const uint64_t rest = want - before;
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    for_row([&](int v, float l) {
      const uint64_t k = cand_key(l, (uint32_t)v);
      if (bin(l) == b && k >= lim) {
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
      for (int i = threadIdx.x; i < 256; i += kSamplePick) s.bins[i] = 0;
      __syncthreads();
      for_row([&](int v, float l) {
        const uint64_t k = cand_key(l, (uint32_t)v);
        if (bin(l) == b && k >= lim && (k & mask) == prefix)
          atomicAdd((unsigned long long*)&s.bins[255 - ((k >> shift) & 255)], MASS ? (unsigned long long)mass(l) : 1ull);
      });
      __syncthreads();
      const int at = block_find(s, 256, left, [&](int i) { return s.bins[i]; }, before);
      prefix |= (uint64_t)(255 - max(at, 0)) << shift;
      mask |= 255ull << shift;
      left -= min(before, left - 1);
      __syncthreads();
    }
    return prefix;
  }

  __device__ __forceinline__ void pick_stream() {
    uint64_t lim = 0;
    if (p.top_k > 0) lim = cut<false>(lim, [&](uint64_t) { return (uint64_t)p.top_k; });
    if (p.top_p < 1.0)
      lim = cut<true>(lim, [&](uint64_t total) { return (uint64_t)fmax(ceil(p.top_p * (double)total), 1.0); });
    const Kept k = kept_from(NAN, lim);
    for (int i = threadIdx.x; i < A.segs; i += kSamplePick) s.bins[i] = 0;
    __syncthreads();
    // a wave's ids of one vector lie in one segment (64 * N divides it)
    for (int v = (int)threadIdx.x * N; v < (A.V + kSampleSeg - 1) / kSampleSeg * kSampleSeg; v += kSamplePick * N) {
      float x[N];
      sample_load<E>(row, v, A.V, x);
      uint64_t a = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (is_kept(k, v + i, x[i])) a += kept_mass(x[i]);
      a = wave_sum(a);
      if ((threadIdx.x & 63) == 0 && a) atomicAdd((unsigned long long*)&s.bins[v / kSampleSeg], (unsigned long long)a);
    }
    __syncthreads();
    draw_segment(k);
  }

  __device__ __forceinline__ void set_max(float largest) {
    m = largest;
    grid = SampleGrid(m, p, kSampleGrid - 2 * kSampleBins);
  }

  __device__ __forceinline__ void pick() {
    const float* smax = A.smax + (int64_t)r * A.segs;
    m = -INFINITY;
    for (int i = threadIdx.x & 63; i < A.segs; i += 64) m = fmaxf(m, smax[i]);
    m = wave_max(m);                               // every wave the same
    if (m == -INFINITY) {                          // nothing to draw from
      if (threadIdx.x == 0) {
        A.token[r] = -1;
        if (A.logprob) A.logprob[r] = -INFINITY;
      }
      return;
    }
    if (p.greedy) return pick_greedy();
    set_max(m);
    const int mode = sample_scan_mode(A, p);
    Kept k = kept_from(NAN, 0);
    if (mode == kScanMass) {
      for (int i = threadIdx.x; i < A.segs; i += kSamplePick) {
        const double v = A.smass[(int64_t)r * A.segs + i];
        s.bins[i] = v > 0.0 ? (uint64_t)rint(v * sample_weight(smax[i], m, p.c64) * scale) : 0;
      }
      __syncthreads();
    } else {
      // how deep the kept ids can lie
      const bool hist = mode == kScanHist && A.hist;
      if (hist && !grid.on) return sample_stream_row<E>(A, m);
      double all = 0.0, ids = 0.0;
      int lo = 0, hi = kSampleBins - 2;
      if (hist) all = join_hist(lo, hi, ids);
      else if (p.top_k > 0) hi = group_bin(p.top_k);
      // (top_p of top_k's ids needs the mass of all of them)
      if (!hist && p.min_p > 0.0 && p.top_p == 1.0)
        hi = min(hi, (int)fmin(-64.0 * log(p.min_p) + 3.0, (double)(kSampleBins - 2)));
      // (a histogram's row takes the list only if it is short: 250 ids cost
      // more than the border's ids alone, 23 us against 21 in one row)
      const int most = hist ? (ids <= 0.75 * kSampleRank ? kSampleRank : 0) : kSampleList;
      const int n = gather(hi, most);
      if (n <= most) {
        if (!hist && p.top_k == 0 && p.top_p < 1.0) {
          uint64_t part = 0;
          for (int i = threadIdx.x; i < n; i += kSamplePick) part += mass(key_logit(s.key[i]));
          all = (double)block_total(s, part);
        }
        return pick_list(n, all);
      }
      if (!hist || !cut_hist(all, lo, hi, k)) return sample_stream_row<E>(A, m);
    }
    draw_segment(k);
  }
};

// The rare path, kept out of the kernel's registers.
template <class E>
__device__ void sample_stream_row(SampleArgs A, float m) {
  SamplePicker<E> pick(A);
  pick.set_max(m);
  pick.pick_stream();
}

// A block per row.  Latency of its steps one after the other for few rows (12
// us for one row of 201088 with top_k and top_p, 30 for 64 bf16 rows of 128256
// with min_p); 256 flat fp32 rows of 201088 with top_p 66 us, most of them for
// reading the row again from the caches.
template <class E>
__global__ __launch_bounds__(kSamplePick) void sample_pick_kernel(SampleArgs A) {
  SamplePicker<E> pick(A);
  pick.pick();
}

}  // namespace kd
