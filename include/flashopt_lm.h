/*
 * flashopt_lm.h -- C ABI of the operators that stand between a language model
 * and the fused steps of flashopt.h: what a loss reads from a model's logits
 * and the BF16 gradient it hands back (log probabilities of given tokens,
 * distillation from a teacher's top logits), and a trained model's weights
 * held in 8 bits (row quantisers, an 8-bit integer linear layer).
 *
 * Conventions are those of flashopt.h: DEVICE pointers owned by the caller,
 * no device memory allocated, streams as void*, host validation before any
 * launch (a failed call launches nothing), no synchronisation, no C++
 * exception.  Every call may be captured into a HIP graph.  A workspace is
 * written and read by its call only: calls that may overlap (other streams,
 * graphs replayed at the same time) need workspaces of their own.  No output
 * may share memory with an input, except a gradient that takes its logits'
 * place; a gradient or layer output that overlaps its logits or input
 * otherwise is refused (FLASHOPT_ERR_ARG).
 */
#ifndef FLASHOPT_LM_H
#define FLASHOPT_LM_H

#include "flashopt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of logits, activations and outputs. */
typedef enum flashopt_type {
    FLASHOPT_BF16 = 0,
    FLASHOPT_FP16 = 1,
    FLASHOPT_FP32 = 2
} flashopt_type;

/* ---- rows of logits -------------------------------------------------------
 *
 * `logits` is rows x vocab, row r at element r * stride (stride >= vocab),
 * aligned to its element type only (rows of an odd vocabulary start
 * anywhere).  With z = x / T (T > 0, the temperature),
 *   m = max_j z_j,  S = sum_j e^(z_j - m),  p_j = e^(z_j - m) / S.
 * An entry of -inf has probability 0 and, unless it is the given token or a
 * listed one, gradient 0 (those keep their own term, gl / T or -g q / T).  A row
 * whose entries are all -inf has no distribution: its entropy and loss are 0, its
 * log probabilities -inf and its gradient 0.  Entries of the type's lowest value
 * are ordinary numbers.  A NaN or +inf in a row gives NaN in that row's
 * results (its top_id stay in range).  Sums are binary32; a gradient is
 * rounded once, to the logits' type, to nearest even.  What lies within a factor
 * of 16 of binary32's largest number (temperatures near 2^-126) may be infinite.
 *
 * A token id outside [0, vocab) stands for none (padding; -100 by custom):
 * its row's log probability is 0 and has no gradient, and a teacher's
 * alternative with such an id is skipped.  Ids are never read out of range.
 *
 * Limits: 0 <= rows <= FLASHOPT_ROWS_MAX (a quarter of that above a vocabulary of
 * 131072), 1 <= vocab <= FLASHOPT_VOCAB_MAX, 0 <= top <= FLASHOPT_TOP_MAX and
 * top <= vocab.
 * Errors: FLASHOPT_ERR_SIZE, FLASHOPT_ERR_NULL, FLASHOPT_ERR_ARG (type,
 * temperature, top), FLASHOPT_ERR_ALIGN (a pointer not aligned to its element
 * type; workspace 256 bytes), FLASHOPT_ERR_WORKSPACE, FLASHOPT_ERR_HIP. */
#define FLASHOPT_ROWS_MAX 8388608
#define FLASHOPT_VOCAB_MAX 524288
#define FLASHOPT_TOP_MAX 64

/* The workspace sizes may be 0 (NULL will do then).
 *
 * Per row: the log probability of targets[r], the entropy
 * -sum_j p_j log p_j, the `top` largest entries (their log probabilities and
 * ids, largest first, equal logits by lowest id), and `stats`, four binary32
 * numbers that the backward call reads.  targets may be NULL (logprob then
 * too); any output may be NULL (top_logprob and top_id both or neither;
 * required when top > 0).  top_logprob, top_id: rows x top. */
size_t flashopt_logprob_workspace_bytes(int32_t type, int64_t rows, int64_t vocab, int32_t top);
int flashopt_logprob(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                     int64_t stride, double temperature, const int64_t* targets, int32_t top,
                     void* workspace, size_t workspace_bytes, float* logprob, float* entropy,
                     float* stats, float* top_logprob, int64_t* top_id, void* stream);
/* The gradient with respect to the logits of
 * sum_r grad_logprob[r] * logprob[r] + grad_entropy[r] * entropy[r]:
 *   grad_j = (1/T) (gl ([j = target] - p_j) - gh p_j (log p_j + H)),
 * from the forward call's stats.  Either upstream gradient may be NULL (0).
 * grad: rows x vocab of the logits' type, row stride grad_stride; it may be
 * the logits themselves (with their stride), which it then replaces. */
int flashopt_logprob_backward(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                              int64_t stride, double temperature, const int64_t* targets,
                              const float* stats, const float* grad_logprob,
                              const float* grad_entropy, void* grad, int64_t grad_stride,
                              void* stream);
/* Both in one call, for upstream gradients known beforehand (a mean of
 * negative log probabilities: grad_logprob = -1/rows). */
int flashopt_logprob_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                          int64_t stride, double temperature, const int64_t* targets,
                          const float* grad_logprob, const float* grad_entropy, void* workspace,
                          size_t workspace_bytes, float* logprob, float* entropy, void* grad,
                          int64_t grad_stride, void* stream);

/* Distillation.  A teacher gives each row `top` token ids and their log
 * probabilities t_k at the same temperature (flashopt_logprob's top_id and
 * top_logprob); 1 <= top.  q_k = e^(t_k) over the ids in range.
 *   tail = 0: q is divided by its sum (t may lie anywhere: scores will do);
 *             loss = sum_k q_k (log q_k - log p_k);
 *   tail = 1: the rest of the vocabulary is one more outcome, with
 *             r = max(0, 1 - sum q) and P = sum of p_j over the ids not
 *             listed: loss += r (log r - log P); where P = 0 (nothing is
 *             left outside the list) the rest is dropped.
 * An id listed twice counts twice in the sums over k and once in P.  With
 * Q = sum_k q_k the gradient with respect to the logits is
 *   grad_j = (g/T) (p_j (Q + r) - sum_{k: id_k = j} q_k - [j not listed] r p_j / P),
 * g = grad_loss[r] (scale it by T^2 for the customary weight).  A row with no
 * id in range has loss and gradient 0.  The workspace and stats (eight
 * binary32 numbers a row) serve as above; loss may be NULL. */
size_t flashopt_distill_workspace_bytes(int32_t type, int64_t rows, int64_t vocab);
int flashopt_distill(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                     int64_t stride, double temperature, const int64_t* top_id,
                     const float* top_logprob, int32_t top, int32_t tail, void* workspace,
                     size_t workspace_bytes, float* loss, float* stats, void* stream);
int flashopt_distill_backward(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                              int64_t stride, double temperature, const int64_t* top_id,
                              const float* top_logprob, int32_t top, const float* stats,
                              const float* grad_loss, void* grad, int64_t grad_stride,
                              void* stream);
int flashopt_distill_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                          int64_t stride, double temperature, const int64_t* top_id,
                          const float* top_logprob, int32_t top, int32_t tail,
                          const float* grad_loss, void* workspace, size_t workspace_bytes,
                          float* loss, void* grad, int64_t grad_stride, void* stream);

/* ---- 8-bit rows -------------------------------------------------------------
 *
 * A matrix of rows x cols in 8 bits: codes row r at byte r * ld with
 * ld = flashopt_int8_ld(cols) (cols rounded up to 128, the padding holding
 * zeros), and one binary32 scale a row.  With a = max_c |x_c| of the row,
 *   q_c = rne(127 x_c / a) in [-127, 127],  scale = RN(a / 127),
 * the quotient decided as if exact; a row of zeros has codes and scale 0.  A
 * row holding an infinity or NaN has codes 0 and scale NaN, so that all that
 * is computed from it is NaN.  Codes are 16-byte aligned, scales 4.
 * Limits: rows <= 2^24, cols <= FLASHOPT_INT8_COLS_MAX (so that a sum of products
 * fits a 32-bit integer); a product (m/128 + 1)(n/128 + 1) <= 2^30. */
#define FLASHOPT_INT8_COLS_MAX 131072
int64_t flashopt_int8_ld(int64_t cols);
/* From rows x cols values of `type`, row stride `stride` elements. */
int flashopt_quantize_rows(const void* x, int32_t type, int64_t rows, int64_t cols,
                           int64_t stride, int8_t* codes, float* scale, void* stream);
/* From one tensor's state (any kind): its master weight theta' + (rho*K8)*h
 * (or the FP32 master weight) as numel / cols rows, rebuilt twice (for a row's scale, then
 * for its codes) without an FP32 copy.  cols must divide numel. */
int flashopt_tensor_quantize_rows(const flashopt_tensor* t, int32_t kind, int64_t cols,
                                  int8_t* codes, float* scale, void* stream);
/* out[i][j] = RN_type(a_scale[i] * b_scale[j] * sum_c a[i][c] b[j][c] + bias[j]):
 * a is m x k (tokens), b n x k (output channels), both as above; bias (of
 * out_type) may be NULL; out row i at element i * out_stride, out_stride >= n.
 * The sum is an exact 32-bit integer; the scales' product is formed first, in
 * binary32. */
size_t flashopt_int8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k);
int flashopt_int8_matmul(const int8_t* a, const float* a_scale, const int8_t* b,
                         const float* b_scale, const void* bias, int64_t m, int64_t n, int64_t k,
                         void* out, int32_t out_type, int64_t out_stride, void* workspace,
                         size_t workspace_bytes, void* stream);
/* The linear layer: rows of x (m x k of `type`, row stride x_stride) rounded
 * to 8 bits as above, then the product, out of the same type.  The workspace
 * holds the rounded rows (both sizes may be 0, NULL will do then). */
size_t flashopt_int8_workspace_bytes(int64_t m, int64_t n, int64_t k);
int flashopt_int8_linear(const void* x, int32_t type, int64_t m, int64_t k, int64_t x_stride,
                         const int8_t* w, const float* w_scale, const void* bias, int64_t n,
                         void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FLASHOPT_LM_H */
