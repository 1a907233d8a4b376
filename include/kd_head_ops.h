/*
 * kd_head_ops.h -- C ABI of the operators around the output head on AMD
 * Instinct MI355X (gfx950): the layer norm whose output the head reads, 8-bit
 * checkpoints of activations and their use in the backward passes, the head's
 * logits, and token sampling from them.  Same library, status codes and
 * element types as kd_topk_kl.h.
 *
 * Conventions (those of kd_topk_kl.h):
 *  - Pointers are device memory owned by the caller; nothing is allocated, no
 *    pointer is kept and there is no global state, so calls on different
 *    streams are independent as long as their outputs and workspaces differ.
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream; its
 *    device must be the current one) without synchronising.  Every call may be
 *    captured into a graph.
 *  - Argument errors are returned before anything is enqueued.
 *  - Fixed-order reductions: two calls on the same inputs give the same bits.
 *  - Rows are contiguous along their last dimension; row strides given as
 *    ld* are in elements and at least the row's length.  Pointers need only
 *    the alignment of their elements unless said otherwise.
 */
#ifndef KD_HEAD_OPS_H
#define KD_HEAD_OPS_H

#include "kd_topk_kl.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KD_ERR_BAD_PARAM 10  /* eps, temperature, top_k, top_p or min_p outside its range */

/* Elements of a row that share one scale of an 8-bit checkpoint. */
#define KD_ACT8_BLOCK 128
/* Largest width of kd_layer_norm_*. */
#define KD_NORM_MAX_D 32768
/* Largest vocabulary of kd_head_logits and kd_sample. */
#define KD_HEAD_MAX_V 16777216

/*
 * 8-bit checkpoint of an activation x [T, d].  Per row and block of
 * KD_ACT8_BLOCK elements (the last one of a row may be shorter), in single
 * precision:
 *   s = max(amax * fl(1/127), 2^-126),  q = clamp(rint(x * fl(1/s)), -127, 127)
 * and the value kept is q * s: within amax / 254 of x, up to rounding.  A block
 * that holds an Inf or a NaN has the scale NaN and comes back as NaN.
 *  x      device [T, d], row stride ldx, dtype
 *  q      device [T, d] int8 (written)
 *  scale  device [T, ceil(d / KD_ACT8_BLOCK)] float32 (written)
 * T >= 1, 1 <= d <= 2^24; T <= 2^24.
 */
int32_t kd_act8_quantize(const void* x, int64_t ldx, int32_t dtype, int64_t T, int64_t d, int8_t* q, float* scale,
                         void* stream);
/* Back to values, rounded to dtype: out device [T, d]. */
int32_t kd_act8_dequantize(const int8_t* q, const float* scale, int32_t dtype, int64_t T, int64_t d, void* out,
                           void* stream);

/*
 * Layer norm of the rows of x [T, d]:
 *   mean, rstd = 1 / sqrt(var + eps) (biased variance),
 *   y = (x - mean) rstd weight + bias.
 *  x        device [T, d], row stride ldx, dtype
 *  weight, bias  device [d], w_dtype (KD_F32, or dtype); bias may be NULL
 *  eps      >= 0, finite
 *  y        device [T, d], dtype (written)
 *  mean, rstd  device [T] float32 (written): what the backward reads
 *  q, scale both NULL, or the 8-bit checkpoint of x (kd_act8_quantize) to be
 *           written in the same pass, for a backward that does not keep x
 * 1 <= d <= KD_NORM_MAX_D; 1 <= T <= 2^30.
 */
int32_t kd_layer_norm_fwd(const void* x, int64_t ldx, int32_t dtype, const void* weight, const void* bias,
                          int32_t w_dtype, int64_t T, int64_t d, float eps, void* y, float* mean, float* rstd,
                          int8_t* q, float* scale, void* stream);

/*
 * Its backward.  Exactly one of x and (q, scale) is given: with a checkpoint,
 * x is replaced by the values it stands for (mean and rstd are the forward's).
 *  dy       device [T, d], dtype
 *  dx       device [T, d], dtype (written), or NULL
 *  dweight, dbias  device [d] float32 (written), or NULL each
 * Workspace: kd_layer_norm_bwd_workspace_bytes(T, d) bytes, 256-byte aligned;
 * may be NULL when neither dweight nor dbias is asked for.
 */
size_t kd_layer_norm_bwd_workspace_bytes(int64_t T, int64_t d);
int32_t kd_layer_norm_bwd(const void* dy, const void* x, int64_t ldx, const int8_t* q, const float* scale,
                          int32_t dtype, const void* weight, int32_t w_dtype, int64_t T, int64_t d,
                          const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * kd_topk_kl_bwd from an 8-bit checkpoint of hidden: (q, scale) of
 * hidden [T, d] in place of it; each chunk's rows are brought back (rounded
 * to in_dtype) in the workspace.  The gradients are those of the loss with
 * the logits recomputed from these rows and row_lse the forward's.  Workspace
 * kd_topk_kl_bwd_act8_workspace_bytes(...).  Everything else as for
 * kd_topk_kl_bwd.
 */
size_t kd_topk_kl_bwd_act8_workspace_bytes(int64_t T, int64_t d, int64_t V, int64_t K, int64_t chunk,
                                           int32_t in_dtype);
int32_t kd_topk_kl_bwd_act8(const int8_t* q, const float* scale, const void* W, int32_t in_dtype,
                            const int32_t* teacher_idx, const float* teacher_logit, const uint8_t* mask, int64_t T,
                            int64_t d, int64_t V, int64_t K, float tau, int64_t chunk, const float* row_lse,
                            const float* grad_loss, void* grad_hidden, int32_t grad_hidden_dtype, float* grad_W,
                            int32_t accumulate_grad_W, uint16_t* grad_W_bf16, void* workspace, size_t workspace_bytes,
                            int32_t* status_dev, void* stream);

/*
 * Logits of the output head: z[t, v] = hidden[t] . W[v], fp32 sums of exact
 * products.
 *  hidden  device [T, d], row stride ldh, in_dtype
 *  W       device [V, d], in_dtype; 16-byte aligned (KD_ERR_BAD_SHAPE) unless
 *          the call is one of few rows or d is not a multiple of 64
 *  logits  device [T, V] float32 (written)
 * Up to 32 rows (a decoding step; 64 where d is not a multiple of 64) read W
 * once and need no workspace; more rows run on the library's matrix product,
 * whose workspace holds zero-padded copies of the operands where d is not a
 * multiple of 64, and one of hidden where its rows do not start at multiples
 * of 16 bytes: kd_head_logits_workspace_bytes(...), 256-byte aligned, 0 if
 * none is needed (or the sizes are invalid).
 * 1 <= d <= 2^20, 1 <= V <= KD_HEAD_MAX_V, 1 <= T <= 2^24.
 */
size_t kd_head_logits_workspace_bytes(int64_t T, int64_t d, int64_t V, int32_t in_dtype);
int32_t kd_head_logits(const void* hidden, int64_t ldh, const void* W, int32_t in_dtype, int64_t T, int64_t d,
                       int64_t V, float* logits, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token id per row of logits [R, V], from a uniform number per row.
 * Per row, ids ordered by (logit descending, id ascending), probabilities
 * those of softmax(logits / temperature):
 *   top_k  keeps the first top_k ids (0: all);
 *   top_p  keeps the shortest prefix of these whose mass is >= top_p of
 *          theirs (1: all);
 *   min_p  keeps those of these with p >= min_p * p_max (0: all);
 * and the drawn id is the first in id order whose inclusive mass exceeds u
 * times the kept mass.  temperature 0 takes the largest logit (lowest id).
 * -inf and NaN logits are never drawn; a row that has no others gets the
 * token -1 and the log-probability -inf.  Borders are decided in 64 bits; an
 * id whose probability is below 1.3e-14 of the largest may count as zero.
 *  logits  device [R, V], row stride ldz, dtype
 *  u       device [R] float32 or (u_is_f64) float64, in [0, 1); values
 *          outside are taken as the nearest end, NaN as 0
 *  temperature >= 0 and finite, top_k >= 0, 0 < top_p <= 1, 0 <= min_p <= 1:
 *          for all rows; or per row from device arrays (each may be NULL):
 *  temperature_rows, top_p_rows, min_p_rows  device [R] float64
 *  top_k_rows  device [R] int32; values of these arrays outside the ranges
 *          above switch the filter off, except that a temperature <= 0 or NaN
 *          takes the largest logit, top_p <= 0 keeps the first id and
 *          min_p > 1 those equal to the largest
 *  token   device [R] int32 (written)
 *  logprob device [R] float32 (written) or NULL: ln of the probability with
 *          which the token was drawn (after the filters)
 * Workspace: kd_sample_workspace_bytes(R, V) bytes, 256-byte aligned.
 */
size_t kd_sample_workspace_bytes(int64_t R, int64_t V);
int32_t kd_sample(const void* logits, int64_t ldz, int32_t dtype, int64_t R, int64_t V, const void* u,
                  int32_t u_is_f64, double temperature, int64_t top_k, double top_p, double min_p,
                  const double* temperature_rows, const int32_t* top_k_rows, const double* top_p_rows,
                  const double* min_p_rows, int32_t* token, float* logprob, void* workspace, size_t workspace_bytes,
                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KD_HEAD_OPS_H */
