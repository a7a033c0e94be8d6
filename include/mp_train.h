/*
 * mp_train.h — C ABI of libmpadamw.so, second part: the operators at the head
 * of a bf16 training step, whose gradients the optimizer step of mp_adamw.h
 * takes: layer norm, log probabilities of given tokens, and distillation from
 * a teacher's top logits, each with its backward pass.
 *
 * The conventions of mp_adamw.h hold: device pointers owned by the caller,
 * every call only enqueues work on `stream`, arguments are checked on the
 * host before any launch, nothing is allocated, statuses as there. Further:
 *  - Matrices are row-major with their last dimension contiguous; `*_stride`
 *    is the distance between rows in elements, at least the row's length, so
 *    a row range or a column range of a wider buffer can be passed.
 *  - A matrix's element type is an mp_dtype_t. Values are widened to fp32,
 *    every sum, mean, maximum and exponential is held in fp32 or more, and
 *    a result is rounded to nearest even once, when it is written.
 *  - Results are bit-identical on every run with the same arguments, sizes
 *    and alignments on the same GPU model (no float atomics).
 *  - Waits inside a kernel end after a second at most. Should one run out (a
 *    fault of the GPU), layer norm's outputs are NaN from there on; what
 *    distillation leaves is said there.
 *  - Any row count, length, stride and element-aligned address is accepted.
 *    Rows that start on 16-B boundaries and hold a multiple of 16 bytes run
 *    wide loads and stores; others run narrower ones, slower.
 */
#ifndef MP_TRAIN_H
#define MP_TRAIN_H

#include "mp_adamw.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mp_dtype {
    MP_BF16 = 0,
    MP_FP16 = 1,
    MP_FP32 = 2
} mp_dtype_t;

typedef enum mp_index_type {
    MP_INT32 = 0,
    MP_INT64 = 1
} mp_index_type_t;

/* ---------------------------------------------------------------------------
 * Layer norm, forward. Per row x of d values:
 *
 *   mean = sum(x) / d;   var = sum((x - mean)^2) / d;   rstd = 1 / sqrt(var + eps)
 *   y[j] = (x[j] - mean) * rstd * weight[j] + bias[j]
 *
 *   y           [rows, d] of `type`, written; may be x itself (same stride).
 *   mean, rstd  float[rows], written for the backward pass; may be NULL.
 *   x           [rows, d] of `type`.
 *   weight      [d] of `weight_type`; NULL: ones.
 *   bias        [d] of `weight_type`; NULL: zeros.
 *   rows >= 0 (0 is a no-op), d in [1, 2^24], eps finite and >= 0.
 * Errors: MP_ERR_NULL, MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
int mp_layernorm_forward(void* y, float* mean, float* rstd, const void* x, const void* weight, const void* bias,
                         int64_t rows, int64_t d, int64_t y_stride, int64_t x_stride, float eps,
                         int32_t type, int32_t weight_type, void* stream);

/* ---------------------------------------------------------------------------
 * Layer norm, backward. With xh = (x - mean) * rstd and g = dy * weight:
 *
 *   dx[j]      = rstd * (g[j] - sum(g) / d - xh[j] * sum(g * xh) / d)     per row
 *   dweight[j] = sum over rows of dy[j] * xh[j]
 *   dbias[j]   = sum over rows of dy[j]
 *
 *   dx          [rows, d] of `type`, written; may be dy itself (same stride);
 *               NULL: not wanted.
 *   dweight, dbias   [d] of `weight_type` (for instance ranges of the flat
 *               bf16 gradient buffer), written, not added to; either may be
 *               NULL. The sums over rows are held in fp32, added in a fixed
 *               order and rounded once. With rows = 0 they are zero.
 *   dy, x       [rows, d] of `type`.
 *   weight      [d] of `weight_type`; NULL: ones.
 *   mean, rstd  float[rows], the forward pass's.
 *   workspace   device scratch of at least mp_layernorm_workspace_bytes(rows, d)
 *               bytes, 16-B aligned, not shared with another call in flight;
 *               may be NULL when neither dweight nor dbias is wanted.
 *   rows, d     as the forward pass.
 * Errors: MP_ERR_NULL, MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_WORKSPACE,
 *         MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
size_t mp_layernorm_workspace_bytes(int64_t rows, int64_t d);

int mp_layernorm_backward(void* dx, void* dweight, void* dbias, const void* dy, const void* x, const void* weight,
                          const float* mean, const float* rstd, int64_t rows, int64_t d, int64_t dx_stride,
                          int64_t dy_stride, int64_t x_stride, int32_t type, int32_t weight_type,
                          void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Log probabilities of given tokens, with entropy and top alternatives. Per
 * row of logits x, with z = scale * x (scale = 1 / temperature):
 *
 *   lse     = log(sum_j exp(z[j]))
 *   logp    = z[target] - lse             (cross entropy is -logp)
 *   entropy = -sum_j p[j] log p[j],       p[j] = exp(z[j] - lse)
 *   top     the top_k largest logits in falling order, equal ones by rising
 *           index: their indices and log probabilities
 *
 *   logp        float[rows], written; NULL exactly when targets is NULL.
 *   lse, entropy   float[rows], written; may be NULL.
 *   top_logp    float[rows, top_k], top_index int32[rows, top_k], written;
 *               NULL when top_k is 0.
 *   logits      [rows, vocab] of `type`, row distance `stride`.
 *   targets     [rows] of `index_type`; negative: no given token (logp 0).
 *               A target >= vocab gives logp NaN and stores MP_ERR_RANGE into
 *               *d_status (if it held 0); nothing is read out of range.
 *   rows >= 0 (0 is a no-op), vocab in [1, 2^31 - 1], 0 < scale <= 2^126,
 *   0 <= top_k <= min(32, vocab).
 *   d_status    int32[1], may be NULL.
 * Masked tokens have logit -inf: probability 0, and no part in the entropy.
 * A row that is -inf throughout has lse -inf, logp -inf and entropy 0. A row
 * that holds NaN or +inf has lse, logp, entropy and top_logp NaN; in the order
 * of the alternatives NaN ranks above +inf. Differences of a row's logits are
 * fp32: more than 3.4e38 below the largest counts as -inf.
 * Errors: MP_ERR_NULL, MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
int mp_token_logprob_forward(float* logp, float* lse, float* entropy, float* top_logp, int32_t* top_index,
                             const void* logits, const void* targets, int64_t rows, int64_t vocab, int64_t stride,
                             float scale, int32_t top_k, int32_t type, int32_t index_type, int32_t* d_status,
                             void* stream);

/* ---------------------------------------------------------------------------
 * Its backward pass: the gradient of the logits for the gradients dlogp of
 * logp and dentropy of entropy, from the forward pass's lse and entropy:
 *
 *   dlogits[j] = scale * ( dlogp * ([j = target] - p[j])
 *                          - dentropy * p[j] * (log p[j] + entropy) )
 *
 *   dlogits     [rows, vocab] of `type`, written; may be logits itself (same
 *               stride).
 *   logits, targets, rows, vocab, scale, type, index_type, d_status   as the
 *               forward pass; a row whose target is negative or >= vocab (or
 *               every row, if targets and dlogp are NULL) takes dlogp as 0.
 *   lse         float[rows], the forward pass's.
 *   dlogp       float[rows]; NULL exactly when targets is NULL.
 *   entropy, dentropy   float[rows] both, or both NULL (dentropy 0).
 * A row whose dlogp and dentropy are both 0, or whose lse is -inf, gets a
 * zero gradient. p is taken from lse, whose fp32 rounding (2^-24 |lse|) is a
 * relative error of the row's every p: a row that is masked throughout should
 * hold -inf, not a finite value of large magnitude.
 * Errors: MP_ERR_NULL (also when there is neither dlogp nor dentropy),
 *         MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
int mp_token_logprob_backward(void* dlogits, const void* logits, const void* targets, const float* lse,
                              const float* entropy, const float* dlogp, const float* dentropy, int64_t rows,
                              int64_t vocab, int64_t dlogits_stride, int64_t stride, float scale, int32_t type,
                              int32_t index_type, int32_t* d_status, void* stream);

/* ---------------------------------------------------------------------------
 * Distillation from a teacher's top logits: loss and gradient in one call.
 * Per row, with the teacher's k listed tokens index[i] and logits teacher[i]:
 *
 *   q[i]  = exp(scale * teacher[i]) / sum_i exp(scale * teacher[i])
 *   p     = softmax(scale * logits) over the whole vocabulary
 *   loss  = row_weight * sum_i q[i] * (log q[i] - log p[index[i]])
 *   dlogits[j] = row_weight * scale * (p[j] - sum of q[i] with index[i] = j)
 *
 * (scale = 1 / temperature; the usual factor temperature^2 and the mean over
 * rows go into row_weight. With k = 1 the loss is cross entropy.)
 *
 *   loss        float[rows], written.
 *   dlogits     [rows, vocab] of `type`, written; may be logits itself (same
 *               stride); NULL: the loss alone.
 *   logits      [rows, vocab] of `type`, row distance `stride`.
 *   teacher     [rows, k] of `type`, row distance teacher_stride.
 *   index       [rows, k] of `index_type`, row distance index_stride; negative
 *               entries are unused (shorter lists). A token may be listed more
 *               than once; its probabilities add up. An index >= vocab is
 *               unused too, and makes the row's loss NaN and stores
 *               MP_ERR_RANGE into *d_status (if it held 0).
 *   row_weight  float[rows], or NULL: ones. A row of weight 0 has loss 0 and a
 *               zero gradient, whatever its logits hold.
 *   rows >= 0 (0 is a no-op), vocab in [1, 2^31 - 1], k in [1, 1024],
 *   0 < scale <= 2^126.
 * A teacher logit of -inf has q = 0 and adds nothing. A row without a listed
 * token of q > 0 has loss 0 and a zero gradient. A listed token of q > 0
 * whose student logit is -inf makes the loss +inf. A student row that is
 * -inf throughout has a zero gradient. NaN or +inf among a row's logits
 * makes its loss and gradient NaN, among its listed teacher logits the loss
 * and the gradient of the listed tokens.
 * Should a wait inside the kernel run out (after a second; a fault of the GPU),
 * every row that is not whole has loss NaN and dlogits[r][0] NaN, and
 * MP_ERR_CUDA is stored into *d_status (if it held 0).
 * Errors: MP_ERR_NULL, MP_ERR_ALIGN, MP_ERR_RANGE, MP_ERR_CUDA.
 * ------------------------------------------------------------------------- */
int mp_distill_topk(float* loss, void* dlogits, const void* logits, const void* teacher, const void* index,
                    const float* row_weight, int64_t rows, int64_t vocab, int32_t k, int64_t dlogits_stride,
                    int64_t stride, int64_t teacher_stride, int64_t index_stride, float scale, int32_t type,
                    int32_t index_type, int32_t* d_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MP_TRAIN_H */
