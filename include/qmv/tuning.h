/*
 * qmv/tuning.h -- C ABI of libqmv.so, continued: fine-tuning over frozen 4-bit
 * weights, and serving what comes of it.  Low-rank adapters beside a 4-bit
 * projection (forward and backward), and two losses over a 4-bit vocabulary
 * projection whose logits are never kept whole (softmax cross entropy, and the
 * divergence from a teacher's largest logits), each with its gradient.
 *
 * The conventions of qmv.h hold here too: every array is the caller's, device
 * arrays are 16-byte aligned, work is enqueued on ``stream`` and nothing
 * synchronizes the host, and every argument the host can see is checked
 * before anything is launched.  What only the device sees (adapter numbers,
 * targets, a teacher's rows) is checked by the kernels: a value out of range
 * never reaches memory, and what it means is stated at each call.  Nothing is
 * summed by atomics: results repeat bit for bit.  Inputs must be finite; one
 * that is not spoils its own token's outputs (and its adapter's gradients), no
 * other token's; an adapter that is not, its own tokens'.  Outputs must not overlap inputs, the workspace or each other.
 *
 * Sizes: T below 2^30 (lora_4bit_backward: 2^22), columns below 2^22, rows below 2^31 (with adapters 2^22),
 * else QMV_ERR_UNSUPPORTED.  A workspace may hold anything, is 16-byte aligned
 * and as large as its size query says for the call's sizes (QMV_ERR_WORKSPACE);
 * calls that overlap must not share one.
 */
#ifndef QMV_TUNING_H
#define QMV_TUNING_H

#include "../qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A quantized weight [rows, cols]: the arrays of qmv_quantize_4bit (and of
 * qmv_double_quant).  cols is a multiple of 32 and of blocksize, else
 * QMV_ERR_UNSUPPORTED. */
typedef struct {
  const uint8_t *packed;
  qmv_absmax scales;
  int64_t rows;
  int64_t cols;
  int32_t blocksize;
  qmv_quant_type quant_type;
} qmv_weight_4bit;

/*
 * Adapters beside a projection [N, K], all of one rank (smaller ones are
 * padded with zeros):
 *   down   [count, rank, K] device, of the activations' type
 *   up     [count, N, rank] device, of the activations' type
 *   scale  [count] device fp32
 *   count  1 .. 4096, else QMV_ERR_UNSUPPORTED;  rank  a multiple of 8 in [8, 128], else QMV_ERR_UNSUPPORTED
 */
typedef struct {
  const void *down;
  const void *up;
  const float *scale;
  int32_t count;
  int32_t rank;
} qmv_lora;

/*
 * lora_4bit: with a = index[t],
 *   y[t] = W_hat x[t] + bias + up[a] (scale[a] down[a] x[t]),
 * rounded once to y_dtype; a token whose index is outside [0, count) has no
 * adapter.  The projection's operands are those of qmv_gemv_4bit and
 * qmv_gemm_4bit (the table's values or the weights rounded to dtype, see
 * cross_entropy_4bit); the adapter's part is computed from its operands as they are, with
 * sums in fp32.  For more than 64 tokens the inner values, scale[a] down[a] x[t], are
 * carried into the second product as two 16-bit terms: off by 2^-16 of themselves
 * for bf16.  For fp16 both terms are held times a power of two chosen by the token's
 * largest inner value: off by 2^-22 of themselves or 2^-39 of that largest one, whichever is
 * more, where that is between 2^-64 and 2^92.
 *   x      [T, K] device, dtype bf16 or fp16 (fp32: QMV_ERR_UNSUPPORTED)
 *   index  [T] device int32, 4-byte aligned
 *   bias   NULL or [N] in dtype
 *   y      [T, N] device, y_dtype: dtype or fp32
 */
size_t qmv_lora_4bit_workspace(int64_t T, int64_t N, int64_t K, int32_t blocksize, int32_t count,
                               int32_t rank);
int qmv_lora_4bit(const void *x, qmv_dtype dtype, int64_t T, const qmv_weight_4bit *w,
                  const qmv_lora *lora, const int32_t *index, const void *bias, void *y,
                  qmv_dtype y_dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * lora_4bit_backward: the gradients of lora_4bit's x, down and up from that of
 * y, with u = scale down x and v = scale up^T dy of each token:
 *   dx[t] = W_hat^T dy[t] + down[a]^T v[t]
 *   d_down[a] = sum of v[t] x[t]^T,  d_up[a] = sum of dy[t] u[t]^T   over the
 * tokens of adapter a (zeros for an adapter without tokens).  u and v are two 16-bit
 * terms in every product here, for any T, as in lora_4bit; in fp16 sums over an adapter's
 * tokens take them off by 2^-22 of themselves or 2^-37 of the adapter's largest.
 *   dy     [T, N], x [T, K] device, dtype bf16 or fp16; N a multiple of 32
 *          (QMV_ERR_UNSUPPORTED)
 *   dx     [T, K] device, dtype
 *   d_down [count, rank, K], d_up [count, N, rank] device, grad_dtype: dtype
 *          or fp32.  Sums are fp32 and rounded once.
 */
size_t qmv_lora_4bit_backward_workspace(int64_t T, int64_t N, int64_t K, int32_t blocksize,
                                        int32_t count, int32_t rank);
int qmv_lora_4bit_backward(const void *dy, const void *x, qmv_dtype dtype, int64_t T,
                           const qmv_weight_4bit *w, const qmv_lora *lora, const int32_t *index,
                           void *dx, void *d_down, void *d_up, qmv_dtype grad_dtype,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * cross_entropy_4bit: with logits l = W_hat x[t] over the V rows of the weight,
 *   loss[t] = log(sum_v exp l_v) - l_target[t],
 * and, where dloss is given, the gradient of sum_t dloss[t] loss[t]:
 *   dx[t] = dloss[t] (sum_v softmax(l)_v W_hat[v] - W_hat[target[t]]).
 * A token whose target is outside [0, V) does not count: its loss is 0, its
 * row of dx is zeros.  The vocabulary is taken in pieces, and tokens 4096 at a
 * time: at no time are there more than 2^26 logits (those of 17 to 64 tokens come in
 * slices of the sum, which count here each).
 *   x       [T, K] device, dtype bf16 or fp16 (fp32: QMV_ERR_UNSUPPORTED)
 *   target  [T] device int64, 8-byte aligned
 *   dloss   NULL or [T] device fp32;  dx  NULL or [T, K] device, dtype: both or neither
 *   loss    [T] device, loss_dtype: dtype or fp32
 * Products have the operands of qmv_gemm_4bit and qmv_gemm_4bit_backward, with sums
 * in fp32: weights rounded to dtype, or, in the kernels for up to 64 tokens' logits,
 * the table's values rounded to dtype and the block's scale applied in fp32 (one
 * rounding of the weight either way).  Maxima, sums and the target's part of the gradient are fp32,
 * exp(l - max) is rounded to dtype for the second product.
 */
size_t qmv_cross_entropy_4bit_workspace(int64_t T, int64_t V, int64_t K, int32_t blocksize, int32_t grad);
int qmv_cross_entropy_4bit(const void *x, qmv_dtype dtype, int64_t T, const qmv_weight_4bit *w,
                           const int64_t *target, const float *dloss, void *loss,
                           qmv_dtype loss_dtype, void *dx, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * distill_4bit: the divergence from the distribution p of a teacher's k
 * largest logits.  With z = teacher[t] / temperature over the entries whose id
 * is in [0, V), p = softmax(z) and q = softmax(W_hat x[t] / temperature):
 *   loss[t] = sum_j p_j (log p_j - log q_ids[j])
 *   dx[t]   = dloss[t] / temperature (sum_v q_v W_hat[v] - sum_j p_j W_hat[ids[j]]).
 * An entry of -inf has p = 0.  A token without an entry of finite logit has loss 0
 * and zeros in dx.  An id that comes twice is two entries: in the loss each has its
 * own log p_j, so that this is less than the divergence from the distribution with
 * their p summed to P (by the sum of p_j log(P / p_j)), and may be negative; the
 * gradient is the same.  For the divergence the ids of a token have to differ.
 *   ids      [T, k] device int64, 8-byte aligned;  teacher [T, k] device, any type
 *   k        1 .. 128 (QMV_ERR_UNSUPPORTED);  temperature finite, > 0
 * The rest as for cross_entropy_4bit.
 */
size_t qmv_distill_4bit_workspace(int64_t T, int64_t V, int64_t K, int32_t blocksize, int32_t k, int32_t grad);
int qmv_distill_4bit(const void *x, qmv_dtype dtype, int64_t T, const qmv_weight_4bit *w,
                     const int64_t *ids, const void *teacher, qmv_dtype teacher_dtype, int32_t k,
                     float temperature, const float *dloss, void *loss, qmv_dtype loss_dtype,
                     void *dx, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* QMV_TUNING_H */
