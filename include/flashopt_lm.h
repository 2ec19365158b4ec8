/*
 * flashopt_lm.h -- C ABI of the operators that stand between a language model
 * and the fused steps of flashopt.h: what a loss reads from a model's logits
 * and the BF16 gradient it hands back (log probabilities of given tokens,
 * distillation from a teacher's top logits, policy and preference losses), a
 * trained model's weights held in 8 bits (row quantisers, an 8-bit integer
 * linear layer), a layer's activations held in 8 bits between its passes and
 * the gradients from them, and an embedding table's rows and gradient.
 *
 * Conventions are those of flashopt.h: DEVICE pointers owned by the caller,
 * no device memory allocated, streams as void*, host validation before any
 * launch (a failed call launches nothing), no synchronisation, no C++
 * exception.  Every call may be captured into a HIP graph.  A workspace is
 * written and read by its call only: calls that may overlap (other streams,
 * graphs replayed at the same time) need workspaces of their own.  No output
 * may share memory with an input, except a gradient that takes its logits'
 * place; a gradient or layer output that overlaps its logits or input
 * otherwise is refused (FLASHOPT_ERR_ARG), and so is one that overlaps held arrays, a
 * table or its ids, and held arrays that overlap what they are held from.  (Of arrays of
 * one number a row or token nothing is checked.)
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

/* Policy training.  A row's given token (targets[r]) has log probability l, had
 * old_logprob[r] when it was generated and ref_logprob[r] under a reference (NULL: no
 * such term); with rho = e^(l - old), A = advantage[r], t = ref - l, and H the
 * row's entropy,
 *   loss = w (-min(rho A, c(rho) A) + kl (e^t - t - 1) - entropy_weight H),
 * c(rho) = min(max(rho, 1 - clip_low), 1 + clip_high) and w = weight[r] (NULL: 1).  Where
 * A is 0 the first term is; where c(rho) A is the smaller product it has no gradient
 * (at rho on a bound it has).
 * A row without a given token or of weight 0 has loss and gradient 0, whatever its
 * other numbers (and its logits); so has a row without a distribution.
 * 0 <= clip_low <= 1, clip_high >= 0 (infinite: no bound), kl and
 * entropy_weight finite, kl >= 0; kl > 0 needs ref_logprob (else FLASHOPT_ERR_ARG).
 *
 * From log probabilities (entropy_weight = 0): loss and grad_logprob, the
 * gradient of sum_r grad_loss[r] * loss[r] (grad_loss NULL: 1); either may be
 * NULL.  mask[r] = 0 stands for a row without a given token (mask NULL: all have
 * one).  0 <= n <= 2^40. */
int flashopt_policy(const float* logprob, const float* old_logprob, const float* advantage,
                    const float* ref_logprob, const float* weight, const uint8_t* mask, int64_t n,
                    double clip_low, double clip_high, double kl, const float* grad_loss,
                    float* loss, float* grad_logprob, void* stream);
/* From logits, in one call: loss, logprob, entropy (each may be NULL) and the
 * gradient of sum_r loss[r] with respect to the logits (grad as in
 * flashopt_logprob_grad).  The workspace may be of 0 bytes. */
size_t flashopt_policy_workspace_bytes(int32_t type, int64_t rows, int64_t vocab);
int flashopt_policy_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                         int64_t stride, double temperature, const int64_t* targets,
                         const float* old_logprob, const float* advantage,
                         const float* ref_logprob, const float* weight, double clip_low,
                         double clip_high, double kl, double entropy_weight, void* workspace,
                         size_t workspace_bytes, float* loss, float* logprob, float* entropy,
                         void* grad, int64_t grad_stride, void* stream);

/* Preferences.  Sequence i is the tokens [offsets[i], offsets[i + 1]) of
 * 2 * pairs sequences, pair p the chosen one 2p and the rejected one 2p + 1.  With
 *   r_i = beta sum (logprob - ref_logprob) over its tokens (divided by their number
 *         where `average`; 0 for none), d = r_2p - r_(2p+1) - margin,
 *   loss_p = (1 - smoothing) log(1 + e^-d) + smoothing log(1 + e^d),
 * a term of weight 0 left out.  Where d is infinite (one sequence is impossible, itself
 * or by the reference) loss and gradient have their limits; where it is NaN (both
 * are) so are they.
 * reward: 2 * pairs, the r_i.  grad_logprob: the gradient of
 * sum_p grad_loss[p] * loss[p] (NULL: 1), one for each of `tokens`, 0 for tokens
 * of no sequence.  A token with mask[t] = 0 does not count, whatever its numbers
 * (mask NULL: all count).  ref_logprob may be NULL (0), as may any output.  offsets
 * do not decrease and end at or before `tokens`; others are never read or written
 * through (they are limited to 0 .. tokens, and a sequence that would end before it
 * begins is empty), but where sequences then overlap the gradients of shared tokens
 * are unspecified.  Sums are binary64, in an order that depends on
 * the sizes alone.
 * 0 <= tokens <= 2^40, 0 <= pairs <= FLASHOPT_PAIRS_MAX; beta and margin finite,
 * 0 <= smoothing <= 1. */
#define FLASHOPT_PAIRS_MAX 1048576
size_t flashopt_preference_workspace_bytes(int64_t pairs, int64_t tokens);
int flashopt_preference(const float* logprob, const float* ref_logprob, const uint8_t* mask,
                        int64_t tokens, const int64_t* offsets, int64_t pairs, double beta,
                        double margin, double smoothing, int32_t average, const float* grad_loss,
                        void* workspace, size_t workspace_bytes, float* loss, float* reward,
                        float* grad_logprob, void* stream);
/* From logits, in one call: the rows are the tokens, a row without a given token
 * does not count.  loss, reward, logprob (rows) may be NULL; grad as in
 * flashopt_logprob_grad. */
size_t flashopt_preference_grad_workspace_bytes(int32_t type, int64_t rows, int64_t vocab,
                                                int64_t pairs);
int flashopt_preference_grad(const void* logits, int32_t type, int64_t rows, int64_t vocab,
                             int64_t stride, double temperature, const int64_t* targets,
                             const float* ref_logprob, const int64_t* offsets, int64_t pairs,
                             double beta, double margin, double smoothing, int32_t average,
                             const float* grad_loss, void* workspace, size_t workspace_bytes,
                             float* loss, float* reward, float* logprob, void* grad,
                             int64_t grad_stride, void* stream);

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

/* ---- activations held in 8 bits ---------------------------------------------------
 *
 * What a layer keeps between its forward and its backward pass: a matrix of rows x
 * cols as codes, row r at byte r * ld with ld = flashopt_held_ld(cols) (cols rounded
 * up to 128), and a byte for each 32 codes of a row (ld / 32 a row).  A group with
 * a = max |x| holds e, the least exponent with rne(a 2^-e) <= 127, and
 *   q = rne(x 2^-e) in [-127, 127],  value = q 2^e,  byte = e + 127,
 * with -126 <= e <= 121 (FP16: -24 <= e <= 9; at the upper bound q is limited to 127).  So a
 * value is off by at most 2^(e-1), or, where q is limited (FP16 beyond 65280, FP32 beyond
 * 255 * 2^120), by less than 2^e; in either case by at most 1/127 of the group's largest
 * magnitude, unless that is below 2^-120, where e = -126 and it is off by up to 2^-127 (FP16 at
 * e = -24 by nothing).  It is exact in the input's type and in BF16.  A group that holds an
 * infinity or NaN has codes 0 and byte 255: its values read as NaN.  Padding holds
 * zeros.  Codes are 16-byte aligned.
 * Limits: rows <= 2^24, 1 <= cols <= FLASHOPT_INT8_COLS_MAX. */
int64_t flashopt_held_ld(int64_t cols);
/* From rows x cols values of `type`, row stride `stride` elements. */
int flashopt_hold(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t stride,
                  int8_t* codes, uint8_t* powers, void* stream);
/* The values held, as rows x cols of `type` (the type they were held from, or
 * FP32). */
int flashopt_held_values(const int8_t* codes, const uint8_t* powers, int64_t rows, int64_t cols,
                         void* out, int32_t type, int64_t out_stride, void* stream);
/* A linear layer's gradients from its held input x (m x k, held from `type`) and
 * the gradient dy of its output (m x n of `type`, row stride dy_stride):
 *   weight[j][c] = RN_type(sum_r dy[r][j] x[r][c])   (n x k, row stride weight_stride),
 *   bias[j] = RN_type(sum_r dy[r][j])                (NULL: not wanted).
 * Every product is exact and every sum binary32, in an order that depends on the
 * sizes alone; of an FP32 dy what lies below 2^-133 is left out (numbers below 2^-110 are
 * taken towards zero, off by less than 2^-133, in weight and bias).  m = 0 gives zeros.
 * weight and bias may not overlap dy, the held arrays or each other.
 * Limits: m, n <= 2^24, k as cols above, (n/128 + 1)(k/128 + 1) <= 2^23. */
size_t flashopt_held_weight_grad_workspace_bytes(int32_t type, int64_t m, int64_t n, int64_t k);
int flashopt_held_weight_grad(const void* dy, int32_t type, int64_t m, int64_t n,
                              int64_t dy_stride, const int8_t* codes, const uint8_t* powers,
                              int64_t k, void* weight, int64_t weight_stride, void* bias,
                              void* workspace, size_t workspace_bytes, void* stream);

/* An activation function, gated or not: y = f(gate) * up, or f(gate) with up NULL,
 *   FLASHOPT_SILU: f(g) = g / (1 + e^-g),
 *   FLASHOPT_GELU: f(g) = g / (1 + e^(-2u)), u = sqrt(2/pi) (g + 0.044715 g^3)
 *                  (the form by tanh).
 * The forward call also holds gate (and up) in 8 bits; the backward call
 * forms f, its slope and up from the values held:
 *   dgate = dy f'(gate) up,  dup = dy f(gate).
 * Each is formed in binary32 and rounded once (f of -infinity is NaN; a share f / g
 * below 2^-126, silu's below -87.3, counts as 0).  Row strides are in elements; y may be
 * NULL (only held), and so may, all together, the held arrays (only y).  No
 * output may overlap an input. */
#define FLASHOPT_SILU 0
#define FLASHOPT_GELU 1
int flashopt_gated(const void* gate, const void* up, int32_t type, int32_t kind, int64_t rows,
                   int64_t cols, int64_t gate_stride, int64_t up_stride, void* y,
                   int64_t y_stride, int8_t* gate_codes, uint8_t* gate_powers, int8_t* up_codes,
                   uint8_t* up_powers, void* stream);
int flashopt_gated_backward(const void* dy, int32_t type, int32_t kind, int64_t rows, int64_t cols,
                            int64_t dy_stride, const int8_t* gate_codes,
                            const uint8_t* gate_powers, const int8_t* up_codes,
                            const uint8_t* up_powers, void* dgate, int64_t dgate_stride,
                            void* dup, int64_t dup_stride, void* stream);

/* ---- an embedding table -----------------------------------------------------------
 *
 * out[i] = RN_type(scale * weight[ids[i]]), row i at element i * out_stride; a row of
 * zeros for an id outside [0, vocab).  weight: vocab x dim of `type`, row stride
 * weight_stride.  From 8-bit rows (flashopt_quantize_rows): out of `type`, the code
 * times RN(w_scale * scale).
 * The gradient: grad[v] = RN_type(scale * sum of dy[i] over the i with ids[i] = v),
 * for every v (zeros for a token that no id names); the sum is binary32, in an order
 * that depends on the ids alone.
 * Limits: 0 <= n <= FLASHOPT_EMBED_MAX, 1 <= vocab <= FLASHOPT_VOCAB_MAX, 1 <= dim <=
 * FLASHOPT_INT8_COLS_MAX; scale finite. */
#define FLASHOPT_EMBED_MAX 16777216
int flashopt_embedding(const int64_t* ids, int64_t n, const void* weight, int32_t type,
                       int64_t vocab, int64_t dim, int64_t weight_stride, double scale, void* out,
                       int64_t out_stride, void* stream);
int flashopt_embedding_int8(const int64_t* ids, int64_t n, const int8_t* w, const float* w_scale,
                            int64_t vocab, int64_t dim, double scale, void* out, int32_t type,
                            int64_t out_stride, void* stream);
size_t flashopt_embedding_workspace_bytes(int64_t n, int64_t vocab, int64_t dim);
int flashopt_embedding_backward(const int64_t* ids, int64_t n, const void* dy, int32_t type,
                                int64_t dy_stride, int64_t vocab, int64_t dim, double scale,
                                void* workspace, size_t workspace_bytes, void* grad,
                                int64_t grad_stride, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FLASHOPT_LM_H */
