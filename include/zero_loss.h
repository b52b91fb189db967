/*
 * zero_loss.h: C ABI of the loss operators that make the sharded step's
 * gradients at a language model's head, for AMD Instinct MI355X (gfx950).
 *
 * A head is hidden states h [tokens, dim] times a vocabulary matrix W
 * [vocab, dim]: logits z_tj = <h_t, W_j>. Two losses over it, each with the
 * gradient of both factors, without the logits ever being kept: they are made
 * in pieces of the vocabulary, reduced on the spot (forward), or made again
 * and turned into a piece of the logits' gradient (backward).
 *
 * Cross entropy (zero_linear_xent), target y_t, smoothing e, z-loss c:
 *     lse_t  = log sum_j exp z_tj
 *     loss_t = lse_t - (1-e) z_ty - (e/V) sum_j z_tj + c lse_t^2
 *     g_tj   = u_t [ (1 + 2 c lse_t) exp(z_tj - lse_t) - e/V - (1-e) [j = y_t] ]
 * Distillation (zero_linear_distill), temperature s, the teacher's K entries
 * (i_k, l_k) of row t, p = softmax of l / s over the row's entries:
 *     lse_t  = log sum_j exp(z_tj / s)
 *     loss_t = s^2 [ sum_k p_k (log p_k - z_ti_k / s) + lse_t ]
 *     g_tj   = u_t s [ exp(z_tj / s - lse_t) - sum_{k: i_k = j} p_k ]
 * and for both, with u_t the upstream gradient of loss_t,
 *     dhidden = g W,   dweight = g^T h.
 *
 * A row with nothing to learn from (target == ignore_index; no teacher entry)
 * is empty: loss, lse and saved logits 0, dhidden 0, no part in dweight,
 * whatever its hidden states, upstream gradient or lse hold. A row whose
 * target is neither ignore_index nor in [0, vocab), or that has a teacher
 * index >= vocab, is bad: its loss is NaN, otherwise it is as an empty row;
 * nothing is read or written out of range.
 *
 * Arithmetic: products of the given types' values with fp32 sums on the matrix
 * units; softmax statistics, losses and the sum over the vocabulary of dhidden
 * in fp32. loss and lse are rounded by the size of the row's largest logit over the
 * temperature, and so is what a probability in the gradient is formed from (beyond
 * some 2^20 that is more than the difference of neighbours). g is rounded once to
 * the given type for its products: in bf16 under a scale that keeps the largest
 * |u_t| near 1, in fp16 under one that keeps it near 2^14 (what is below 2^-28 of it
 * then has fewer bits, and none below 2^-38), undone in fp32 before the result is
 * rounded. In fp32 hidden, weight and g are each held as three bf16 parts, all 24
 * bits of every value, and six of the nine part products are summed: what is left
 * out is below 2^-23 of each product. A row with an infinity or a NaN leaves the
 * other rows' losses and dhidden as they are; in fp32 a product with an infinity may
 * be NaN where it would otherwise be infinite. The same call gives the same bits:
 * nothing is summed in an order left to chance.
 *
 * Conventions are those of zero_adam.h: caller-owned device buffers, work
 * enqueued on `stream`, arguments validated before any HIP call, status codes,
 * zero_last_error(). No call allocates, copies to the host or synchronises, so
 * each may be captured into a graph.
 */
#ifndef ZERO_LOSS_H
#define ZERO_LOSS_H

#include "zero_adam.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ZERO_LOSS_F32 = 0, ZERO_LOSS_BF16 = 1, ZERO_LOSS_F16 = 2 } zero_loss_dtype;
typedef enum { ZERO_INDEX_I32 = 0, ZERO_INDEX_I64 = 1 } zero_index_dtype;

/* Largest tokens, vocab, dim and entries per row of one call. */
#define ZERO_LOSS_MAX_TOKENS (1 << 20)
#define ZERO_LOSS_MAX_VOCAB (1 << 24)
#define ZERO_LOSS_MAX_DIM (1 << 16)
#define ZERO_LOSS_MAX_K 1024

/* The head of one call. Rows are contiguous; row strides are in elements. */
typedef struct {
  int64_t tokens;        /* 0 <= tokens <= ZERO_LOSS_MAX_TOKENS */
  int64_t vocab;         /* 1 <= vocab <= ZERO_LOSS_MAX_VOCAB */
  int64_t dim;           /* 1 <= dim <= ZERO_LOSS_MAX_DIM */
  const void* hidden;    /* [tokens, dim]; may be NULL when tokens == 0 */
  int64_t hidden_stride; /* >= dim */
  const void* weight;    /* [vocab, dim] */
  int64_t weight_stride; /* >= dim */
  int32_t dtype;         /* a zero_loss_dtype: of hidden, weight and their gradients */
  int32_t reserved;      /* must be 0 */
} zero_head;

/* Hard targets. */
typedef struct {
  const void* target;     /* tokens values, contiguous */
  int32_t index_dtype;    /* a zero_index_dtype: of target */
  int32_t reserved;       /* must be 0 */
  int64_t ignore_index;   /* a target of this value makes its row empty */
  double label_smoothing; /* in [0, 1), as a float */
  double z_loss;          /* finite as a float, >= 0 */
} zero_xent_params;

/* A teacher's top-K entries. index < 0 is padding, and so is a logit of -inf.
 * Of an index that stands more than once in a row every entry has its own term in the
 * loss, and the gradient has the sum of their probabilities. */
typedef struct {
  const void* index;      /* [tokens, k] */
  const void* logit;      /* [tokens, k], the teacher's logits (or log-probabilities) */
  int64_t index_stride;   /* >= k, elements */
  int64_t logit_stride;   /* >= k, elements */
  int32_t k;              /* 1 <= k <= ZERO_LOSS_MAX_K */
  int32_t index_dtype;    /* a zero_index_dtype */
  int32_t logit_dtype;    /* a zero_loss_dtype */
  int32_t reserved;       /* must be 0 */
  double temperature;     /* > 0, its square neither infinite nor subnormal as floats:
                             1.1e-19 to 1.8e19 */
} zero_distill_params;

/* Gradients: device buffers the caller owns; rows contiguous, strides in
 * elements. dhidden or dweight (not both) may be NULL: it is then not formed.
 * dweight may be a view at any element offset, e.g. of a worker's flat
 * gradient buffer. Every element of a non-NULL gradient is written. */
typedef struct {
  const float* upstream;   /* u: the gradient of each token's loss */
  int64_t upstream_stride; /* elements between tokens; 0 broadcasts one value */
  void* dhidden;           /* [tokens, dim] */
  int64_t dhidden_stride;  /* >= dim */
  void* dweight;           /* [vocab, dim] */
  int64_t dweight_stride;  /* >= dim */
} zero_head_grads;

/* Device workspace bytes of the calls below (want_grad 0: the loss, 1: the
 * gradient). Depends on the head's shape, type, strides and alignment only.
 * The workspace must be 256-byte aligned. Host-only. */
zero_status zero_loss_workspace_bytes(const zero_head* head, int32_t want_grad, size_t* bytes);

/* loss[tokens] and lse[tokens] (fp32). */
zero_status zero_linear_xent(const zero_head* head, const zero_xent_params* p, float* loss,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* The gradient, from the lse that zero_linear_xent gave for the same arguments. */
zero_status zero_linear_xent_grad(const zero_head* head, const zero_xent_params* p,
                                  const float* lse, const zero_head_grads* grads, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* loss[tokens], lse[tokens] (of z / temperature) and the student's logits at
 * the teacher's entries, logit[tokens, k] contiguous (0 at padding), fp32. */
zero_status zero_linear_distill(const zero_head* head, const zero_distill_params* p, float* loss,
                                float* lse, float* logit, void* workspace, size_t workspace_bytes,
                                void* stream);

/* The gradient, from the lse and logit that zero_linear_distill gave for the
 * same arguments. */
zero_status zero_linear_distill_grad(const zero_head* head, const zero_distill_params* p,
                                     const float* lse, const float* logit,
                                     const zero_head_grads* grads, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Errors of all of the above: ZERO_EINVAL for a NULL or misaligned pointer
 * (tensors to their element size), a size, stride or scalar outside the ranges
 * given, an unknown type, reserved != 0, a workspace that is too small, or a
 * written buffer that overlaps another buffer of the call; ZERO_EHIP if a
 * launch fails (launches before it may be enqueued). */

#ifdef __cplusplus
}
#endif

#endif /* ZERO_LOSS_H */
