// kd_head_ops.hip -- host side of the operators around the output head:
// argument checks, variant selection and launches, behind the C ABI declared
// in include/kd_head_ops.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/kd_head_ops.h"
#include "kd_act8.hpp"
#include "kd_launch.hpp"
#include "kd_logits.hpp"
#include "kd_norm.hpp"
#include "kd_pad.hpp"
#include "kd_sample.hpp"

namespace kd {
namespace {

int64_t elem_bytes(int32_t dtype) { return dtype == KD_BF16 ? 2 : 4; }
bool known_dtype(int32_t dtype) { return dtype == KD_BF16 || dtype == KD_F32; }
// every element of the buffer is at a multiple of its size
bool misaligned(const void* p, int64_t bytes) { return (((uintptr_t)p) & (uintptr_t)(bytes - 1)) != 0; }

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------
constexpr int64_t kNormMaxBlocks = 1 << 20;   // forward: rows past it are taken in a loop

template <class T, class WT, int WPR, int NV>
int32_t norm_fwd_launch(const NormFwdArgs& A, hipStream_t st) {
  typedef NormFwdCfg<WPR> C;
  const dim3 grid((unsigned)std::min<int64_t>(cdiv(A.T, C::kRows), kNormMaxBlocks));
  if (A.q) hipLaunchKernelGGL((norm_fwd_kernel<T, WT, WPR, NV, true>), grid, dim3(C::kThreads), 0, st, A);
  else hipLaunchKernelGGL((norm_fwd_kernel<T, WT, WPR, NV, false>), grid, dim3(C::kThreads), 0, st, A);
  KD_LAUNCH_CHECK();
  return KD_OK;
}
template <class T, class WT, int WPR, int NV>
int32_t norm_bwd_launch(const NormBwdArgs& A, hipStream_t st) {
  typedef NormBwdCfg<WPR> C;
  const dim3 grid((unsigned)norm_bwd_blocks(A.T, A.d));
  if (A.q) hipLaunchKernelGGL((norm_bwd_kernel<T, WT, WPR, NV, true>), grid, dim3(C::kThreads), 0, st, A);
  else hipLaunchKernelGGL((norm_bwd_kernel<T, WT, WPR, NV, false>), grid, dim3(C::kThreads), 0, st, A);
  KD_LAUNCH_CHECK();
  return KD_OK;
}

// The narrowest variant that holds a row: NV vectors of 8 elements per lane,
// WPR waves per row.  The backward spreads rows wider than 1024 over two waves
// and more: its accumulators take as many registers as two rows, and with one
// wave per row of 2880 they left room for two waves per SIMD (128K rows of 2880
// from 8 bits: 527 us; with two waves 464 at once and 402 since).
template <class T, class WT>
int32_t norm_fwd(const NormFwdArgs& A, hipStream_t st) {
  if (A.d <= 512) return norm_fwd_launch<T, WT, 1, 1>(A, st);
  if (A.d <= 1024) return norm_fwd_launch<T, WT, 1, 2>(A, st);
  if (A.d <= 2048) return norm_fwd_launch<T, WT, 1, 4>(A, st);
  if (A.d <= 6 * 512) return norm_fwd_launch<T, WT, 1, 6>(A, st);
  if (A.d <= 4096) return norm_fwd_launch<T, WT, 4, 2>(A, st);
  if (A.d <= 8192) return norm_fwd_launch<T, WT, 4, 4>(A, st);
  if (A.d <= 16384) return norm_fwd_launch<T, WT, 16, 2>(A, st);
  return norm_fwd_launch<T, WT, 16, 4>(A, st);
}
template <class T, class WT>
int32_t norm_bwd(const NormBwdArgs& A, hipStream_t st) {
  if (A.d <= 512) return norm_bwd_launch<T, WT, 1, 1>(A, st);
  if (A.d <= 1024) return norm_bwd_launch<T, WT, 1, 2>(A, st);
  if (A.d <= 2048) return norm_bwd_launch<T, WT, 2, 2>(A, st);
  if (A.d <= 6 * 512) return norm_bwd_launch<T, WT, 2, 3>(A, st);
  if (A.d <= 4096) return norm_bwd_launch<T, WT, 4, 2>(A, st);
  if (A.d <= 8192) return norm_bwd_launch<T, WT, 4, 4>(A, st);
  if (A.d <= 16384) return norm_bwd_launch<T, WT, 16, 2>(A, st);
  return norm_bwd_launch<T, WT, 8, 8>(A, st);
}

int32_t norm_check(int32_t dtype, int32_t w_dtype, int64_t T, int64_t d) {
  if (!known_dtype(dtype) || !known_dtype(w_dtype) || (dtype == KD_F32 && w_dtype != KD_F32)) return KD_ERR_DTYPE;
  if (T < 1 || d < 1 || d > KD_NORM_MAX_D || T > (1ll << 30)) return KD_ERR_BAD_SHAPE;
  return KD_OK;
}

// ---------------------------------------------------------------------------
// head logits
// ---------------------------------------------------------------------------
template <class E>
int32_t logits_run(const LogitsPlan& P, const void* hidden, int64_t ldh, const void* W, int64_t T, int64_t d,
                   int64_t V, float* logits, char* ws, hipStream_t st) {
  typedef typename E::T S;
  if (P.skinny) {
    const S *h = (const S*)hidden, *w = (const S*)W;
    auto launch = [&](auto kernel, int waves) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv(V, 16 * waves)), dim3(64 * waves), 0, st, h, ldh, (int)T, w,
                         (int)V, (int)d, logits, V);
    };
    // more waves share a block's hidden rows as these grow: at d = 2880, V =
    // 201088, 32 rows take 234 us with eight waves and 245 with four, 64 rows
    // (a d that the matrix product would need a copy of W for) 278 and 284; one
    // row 204 with four and 212 with eight
    if (T <= 16) launch(skinny_logits_kernel<E, 1, 4>, 4);
    else if (T <= 32) launch(skinny_logits_kernel<E, 2, 8>, 8);
    else launch(skinny_logits_kernel<E, 4, 8>, 8);
    KD_LAUNCH_CHECK();
    return KD_OK;
  }
  auto pad = [&](const S* src, int64_t ld, int64_t rows, S* dst) {
    hipLaunchKernelGGL(pad_kernel<E>, dim3((unsigned)std::min<int64_t>(cdiv(rows * P.d_p, 256), 65536)), dim3(256), 0,
                       st, src, ld, rows, d, dst, P.d_p, rows);
  };
  const S* w = (const S*)W;
  int64_t ldw = d;
  if (P.pad_w) {
    pad(w, d, V, (S*)(ws + P.off_wp));
    KD_LAUNCH_CHECK();
    w = (const S*)(ws + P.off_wp);
    ldw = P.d_p;
  }
  for (int64_t t0 = 0; t0 < T; t0 += P.rows) {
    const int64_t n = std::min<int64_t>(P.rows, T - t0);
    const S* h = (const S*)hidden + t0 * ldh;
    int64_t ld = ldh;
    if (P.pad_h) {
      pad(h, ldh, n, (S*)(ws + P.off_hp));
      KD_LAUNCH_CHECK();
      h = (const S*)(ws + P.off_hp);
      ld = P.d_p;
    }
    const EpiStoreLogits epi{logits + t0 * V, V, (int)V, (int)n};
    const int64_t kbytes = P.d_p * E::kBytes;
    auto launch = [&](auto tile) {
      typedef decltype(tile) TC;
      return launch_gemm<TC, E>(make_shape<TC>(w, ldw, (int)V, h, ld, (int)n, kbytes, 1, 1), epi, st);
    };
    const hipError_t e = P.low ? launch(TileLogitsLow()) : P.tall ? launch(TileLogits()) : launch(TileMain());
    if (e != hipSuccess) return KD_ERR_HIP;
  }
  return KD_OK;
}

bool rows_aligned(const void* p, int64_t ld, int64_t eb) {
  return (((uintptr_t)p) & 15) == 0 && (ld * eb) % 16 == 0 && ld * eb < (1ll << 23);
}

// ---------------------------------------------------------------------------
// sampling
// ---------------------------------------------------------------------------
template <class E>
int32_t sample_run(const SampleArgs& A, hipStream_t st) {
  hipLaunchKernelGGL(sample_scan_kernel<E>, dim3((unsigned)(A.R * A.segs)), dim3(kSampleScan), 0, st, A);
  KD_LAUNCH_CHECK();
  hipLaunchKernelGGL(sample_pick_kernel<E>, dim3((unsigned)A.R), dim3(kSamplePick), 0, st, A);
  KD_LAUNCH_CHECK();
  return KD_OK;
}

}  // namespace
}  // namespace kd

extern "C" {

int32_t kd_act8_quantize(const void* x, int64_t ldx, int32_t dtype, int64_t T, int64_t d, int8_t* q, float* scale,
                         void* stream) {
  if (!x || !q || !scale) return KD_ERR_NULL_ARG;
  if (!kd::known_dtype(dtype)) return KD_ERR_DTYPE;
  if (!kd::act8_fits(T, d) || ldx < d) return KD_ERR_BAD_SHAPE;
  if (kd::misaligned(x, kd::elem_bytes(dtype)) || kd::misaligned(scale, 4)) return KD_ERR_BAD_SHAPE;
  hipStream_t st = (hipStream_t)stream;
  if (dtype == KD_BF16) kd::launch_act8_quantize<uint16_t>((const uint16_t*)x, ldx, T, d, q, scale, st);
  else kd::launch_act8_quantize<float>((const float*)x, ldx, T, d, q, scale, st);
  KD_LAUNCH_CHECK();
  return KD_OK;
}

int32_t kd_act8_dequantize(const int8_t* q, const float* scale, int32_t dtype, int64_t T, int64_t d, void* out,
                           void* stream) {
  if (!q || !scale || !out) return KD_ERR_NULL_ARG;
  if (!kd::known_dtype(dtype)) return KD_ERR_DTYPE;
  if (!kd::act8_fits(T, d)) return KD_ERR_BAD_SHAPE;
  if (kd::misaligned(out, kd::elem_bytes(dtype)) || kd::misaligned(scale, 4)) return KD_ERR_BAD_SHAPE;
  if (dtype == KD_BF16) kd::launch_act8_dequantize<uint16_t>(q, scale, T, d, (uint16_t*)out, d, T, (hipStream_t)stream);
  else kd::launch_act8_dequantize<float>(q, scale, T, d, (float*)out, d, T, (hipStream_t)stream);
  KD_LAUNCH_CHECK();
  return KD_OK;
}

int32_t kd_layer_norm_fwd(const void* x, int64_t ldx, int32_t dtype, const void* weight, const void* bias,
                          int32_t w_dtype, int64_t T, int64_t d, float eps, void* y, float* mean, float* rstd,
                          int8_t* q, float* scale, void* stream) {
  if (!x || !weight || !y || !mean || !rstd || !q != !scale) return KD_ERR_NULL_ARG;
  const int32_t rc = kd::norm_check(dtype, w_dtype, T, d);
  if (rc != KD_OK) return rc;
  if (ldx < d) return KD_ERR_BAD_SHAPE;
  if (!(eps >= 0.f) || !isfinite(eps)) return KD_ERR_BAD_PARAM;
  const int64_t eb = kd::elem_bytes(dtype), wb = kd::elem_bytes(w_dtype);
  if (kd::misaligned(x, eb) || kd::misaligned(y, eb) || kd::misaligned(weight, wb) || kd::misaligned(bias, wb) ||
      kd::misaligned(mean, 4) || kd::misaligned(rstd, 4) || kd::misaligned(scale, 4))
    return KD_ERR_BAD_SHAPE;
  const kd::NormFwdArgs A{x, ldx, weight, bias, eps, T, (int)d, (int)kd::cdiv(d, kd::kActBlock), y, mean, rstd, q, scale};
  hipStream_t st = (hipStream_t)stream;
  if (dtype == KD_F32) return kd::norm_fwd<float, float>(A, st);
  if (w_dtype == KD_F32) return kd::norm_fwd<uint16_t, float>(A, st);
  return kd::norm_fwd<uint16_t, uint16_t>(A, st);
}

size_t kd_layer_norm_bwd_workspace_bytes(int64_t T, int64_t d) {
  if (kd::norm_check(KD_BF16, KD_F32, T, d) != KD_OK) return 0;
  return kd::norm_bwd_workspace(T, d);
}

int32_t kd_layer_norm_bwd(const void* dy, const void* x, int64_t ldx, const int8_t* q, const float* scale,
                          int32_t dtype, const void* weight, int32_t w_dtype, int64_t T, int64_t d,
                          const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!dy || !weight || !mean || !rstd || !q != !scale || !x == !q) return KD_ERR_NULL_ARG;
  if (!dx && !dweight && !dbias) return KD_ERR_NULL_ARG;
  const int32_t rc = kd::norm_check(dtype, w_dtype, T, d);
  if (rc != KD_OK) return rc;
  if (x && ldx < d) return KD_ERR_BAD_SHAPE;
  const int64_t eb = kd::elem_bytes(dtype);
  if (kd::misaligned(dy, eb) || kd::misaligned(x, eb) || kd::misaligned(dx, eb) ||
      kd::misaligned(weight, kd::elem_bytes(w_dtype)) || kd::misaligned(mean, 4) || kd::misaligned(rstd, 4) ||
      kd::misaligned(scale, 4) || kd::misaligned(dweight, 4) || kd::misaligned(dbias, 4))
    return KD_ERR_BAD_SHAPE;
  const bool sums = dweight || dbias;
  if (sums && (!workspace || workspace_bytes < kd::norm_bwd_workspace(T, d) || (((uintptr_t)workspace) & 255)))
    return KD_ERR_WORKSPACE;
  const kd::NormBwdArgs A{dy, x, q, scale, weight, mean, rstd, ldx, T, (int)d, (int)kd::cdiv(d, kd::kActBlock), dx,
                          sums ? (float*)workspace : nullptr};
  hipStream_t st = (hipStream_t)stream;
  int32_t s;
  if (dtype == KD_F32) s = kd::norm_bwd<float, float>(A, st);
  else if (w_dtype == KD_F32) s = kd::norm_bwd<uint16_t, float>(A, st);
  else s = kd::norm_bwd<uint16_t, uint16_t>(A, st);
  if (s != KD_OK || !sums) return s;
  hipLaunchKernelGGL(kd::norm_reduce_kernel, dim3((unsigned)kd::cdiv(2 * d, 64)), dim3(1024), 0, st,
                     (const float*)workspace, (int)kd::norm_bwd_blocks(T, d), (int)d, dweight, dbias);
  KD_LAUNCH_CHECK();
  return KD_OK;
}

size_t kd_head_logits_workspace_bytes(int64_t T, int64_t d, int64_t V, int32_t in_dtype) {
  kd::LogitsPlan p;
  // (covers a hidden whose rows do not start at multiples of 16 bytes)
  if (kd::make_logits_plan(T, d, V, in_dtype, false, &p) != KD_OK) return 0;
  return p.total;
}

int32_t kd_head_logits(const void* hidden, int64_t ldh, const void* W, int32_t in_dtype, int64_t T, int64_t d,
                       int64_t V, float* logits, void* workspace, size_t workspace_bytes, void* stream) {
  if (!hidden || !W || !logits) return KD_ERR_NULL_ARG;
  if (!kd::known_dtype(in_dtype)) return KD_ERR_DTYPE;
  const int64_t eb = kd::elem_bytes(in_dtype);
  kd::LogitsPlan p;
  const int32_t rc = kd::make_logits_plan(T, d, V, in_dtype, kd::rows_aligned(hidden, ldh, eb), &p);
  if (rc != KD_OK) return rc;
  if (!p.skinny && !p.pad_w && (((uintptr_t)W) & 15)) return KD_ERR_BAD_SHAPE;
  if (ldh < d || kd::misaligned(hidden, eb) || kd::misaligned(W, eb) || kd::misaligned(logits, 4)) return KD_ERR_BAD_SHAPE;
  if (p.total && (!workspace || workspace_bytes < p.total || (((uintptr_t)workspace) & 255))) return KD_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  if (in_dtype == KD_BF16) return kd::logits_run<kd::Bf16>(p, hidden, ldh, W, T, d, V, logits, (char*)workspace, st);
  return kd::logits_run<kd::F32>(p, hidden, ldh, W, T, d, V, logits, (char*)workspace, st);
}

size_t kd_sample_workspace_bytes(int64_t R, int64_t V) {
  kd::SamplePlan p;
  return kd::make_sample_plan(R, V, &p) == KD_OK ? p.total : 0;
}

int32_t kd_sample(const void* logits, int64_t ldz, int32_t dtype, int64_t R, int64_t V, const void* u,
                  int32_t u_is_f64, double temperature, int64_t top_k, double top_p, double min_p,
                  const double* temperature_rows, const int32_t* top_k_rows, const double* top_p_rows,
                  const double* min_p_rows, int32_t* token, float* logprob, void* workspace, size_t workspace_bytes,
                  void* stream) {
  if (!logits || !u || !token) return KD_ERR_NULL_ARG;
  if (!kd::known_dtype(dtype)) return KD_ERR_DTYPE;
  kd::SamplePlan p;
  const int32_t rc = kd::make_sample_plan(R, V, &p);
  if (rc != KD_OK) return rc;
  if (ldz < V) return KD_ERR_BAD_SHAPE;
  // (the comparisons refuse NaN)
  if (!(temperature >= 0.0) || !isfinite(temperature) || top_k < 0 || !(top_p > 0.0) || !(top_p <= 1.0) ||
      !(min_p >= 0.0) || !(min_p <= 1.0))
    return KD_ERR_BAD_PARAM;
  if (kd::misaligned(logits, kd::elem_bytes(dtype)) || kd::misaligned(u, u_is_f64 ? 8 : 4) ||
      kd::misaligned(temperature_rows, 8) || kd::misaligned(top_k_rows, 4) || kd::misaligned(top_p_rows, 8) ||
      kd::misaligned(min_p_rows, 8) || kd::misaligned(token, 4) || kd::misaligned(logprob, 4))
    return KD_ERR_BAD_SHAPE;
  if (!workspace || workspace_bytes < p.total || (((uintptr_t)workspace) & 255)) return KD_ERR_WORKSPACE;
  kd::SampleArgs A;
  A.z = logits; A.ldz = ldz; A.R = (int)R; A.V = (int)V;
  A.u = u; A.u_is_f64 = u_is_f64;
  A.temperature = temperature; A.top_p = top_p; A.min_p = min_p;
  A.top_k = (int)(top_k < V ? top_k : 0);
  A.temperature_rows = temperature_rows; A.top_k_rows = top_k_rows;
  A.top_p_rows = top_p_rows; A.min_p_rows = min_p_rows;
  char* ws = (char*)workspace;
  A.groups = (int)p.groups; A.segs = (int)p.segs;
  A.gmax = (float*)(ws + p.off_gmax);
  A.smax = (float*)(ws + p.off_smax);
  A.smass = (double*)(ws + p.off_smass);
  A.hlen = (int*)(ws + p.off_hlen);
  A.hist = p.hist ? (uint64_t*)(ws + p.off_hist) : nullptr;
  A.token = token; A.logprob = logprob;
  hipStream_t st = (hipStream_t)stream;
  return dtype == KD_BF16 ? kd::sample_run<kd::Bf16>(A, st) : kd::sample_run<kd::F32>(A, st);
}

}  // extern "C"
