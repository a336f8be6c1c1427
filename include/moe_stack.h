/*
 * moe_stack.h — C ABI of the operators around the blocks of a sparse stack that trains from token
 * ids on GB300 (sm_103a): the embedding lookup and its gradient, the layer norm and its gradient,
 * dropout from a counter-based generator (alone, and in a residual join that also takes the next
 * layer norm, with the join's gradient), and the router's balance and z losses with their
 * gradient. Same library, statuses and conventions as moe.h and moe_train.h: device pointers,
 * contiguous row-major tensors, 16-byte aligned rows, the caller owns every buffer, nothing
 * allocates, synchronises or reads device data on the host, argument errors come back before
 * anything is enqueued, every call can be captured in a CUDA graph. No result depends on the
 * order of atomics. A workspace belongs to one call until that call has run.
 *
 * One step of a stack of blocks x <- x + scale * dropout(MoE(layer_norm(x))):
 *
 *   x          = moe_embed(tokens);  h = moe_layer_norm(x)
 *   logits, ids, w = moe_route(h)                                  (moe.h)
 *   losses     = moe_balance_loss(logits, ids)
 *   y          = the experts' outputs                              (moe_train.h)
 *   x, h       = moe_dropout_join(x, y)            h: the next block's (or the final) norm
 *
 * and backwards: moe_dropout_join_backward, the experts, moe_route_backward with
 * moe_balance_loss_backward added to its dlogits, moe_layer_norm_backward, moe_embed_backward.
 */
#ifndef MOE_STACK_GB300_H
#define MOE_STACK_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- embedding ------------------------------------------------------------------------
 * tokens[T]: int32 (token_bytes 4) or int64 (8), T >= 1, at most 2^28. table[V, H] in dtype, V >= 1, at
 * most 2^26; H a multiple of 8, at most 2^20. A token outside [0, V) (padding) is a row of zeros
 * and gives no gradient. */

/* out[t] = scale * table[tokens[t]], one rounding. */
moe_status_t moe_embed(const void* tokens, int token_bytes, int T, const void* table, int V, int H,
                       moe_dtype_t dtype, float scale, void* out, cudaStream_t stream);

/* dtable[v] (+)= scale * sum of dx[t] over the tokens t of id v, in fp32 in the order of the
 * tokens (long runs in pieces, in a fixed order) and rounded once to out_dtype (fp32, or bf16
 * when dtype is). accumulate 0: all of dtable is written, zeros for ids that do not occur; 1: added
 * to, and rows of ids that do not occur are not touched. ws: 16-byte aligned. */
moe_status_t moe_embed_workspace_size(int T, int V, int H, size_t* bytes);
moe_status_t moe_embed_backward(const void* dx, const void* tokens, int token_bytes, int T, int V,
                                int H, moe_dtype_t dtype, moe_dtype_t out_dtype, float scale,
                                int accumulate, void* dtable, void* ws, size_t ws_bytes,
                                cudaStream_t stream);

/* ---- layer norm, dropout, the join ----------------------------------------------------
 * Rows of H elements (a multiple of 8, at most 32768), 1 <= T <= 2^30 of them, in dtype. Weights
 * and biases, their gradients, mean and rstd are fp32. */
typedef struct moe_layer {
  int T, H;
  moe_dtype_t dtype;
  float eps;   /* >= 0 */
  float scale; /* dropout and join calls */
} moe_layer_t;

/* Dropout of the elements of a [T, H] tensor: element i (row-major) is dropped where its random
 * 32-bit number is below round(p * 2^32), kept ones are multiplied by 1 / (1 - p) with the p so
 * rounded. The number is word i % 4 of Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw:
 * Parallel random numbers: as easy as 1, 2, 3; 2011) of the counter (i / 4 in 64 bits, stream in
 * 64 bits with site added to the upper word) and the key seed. So the mask is a function of
 * (seed, stream, site, i): it is never stored, and the backward pass computes it again. rng: on the
 * device, so that a captured step can be replayed with another stream. Give every place of a step
 * its own site and every step its own stream. */
typedef struct moe_drop {
  double p;           /* 0 <= p < 1; 0: nothing is dropped and rng may be NULL */
  const int64_t* rng; /* device: {seed, stream} */
  uint32_t site;
} moe_drop_t;

/* out = scale * dropout(x), its own gradient: dx = moe_dropout(dout). out may be x. */
moe_status_t moe_dropout(const moe_layer_t* cfg, const moe_drop_t* drop, const void* x, void* out,
                         cudaStream_t stream);

/* h = (x - mean) * rstd * gamma + beta (beta may be NULL), rstd = (mean of (x - mean)^2 + eps)^-1/2.
 * The variance is taken about the mean, not as a difference of squares. */
moe_status_t moe_layer_norm(const moe_layer_t* cfg, const void* x, const float* gamma,
                            const float* beta, void* h, float* mean, float* rstd,
                            cudaStream_t stream);

/* dx = dres + d norm / dx (dres, the gradient that reaches x past the norm, may be NULL),
 * dgamma[H] = sum over tokens of dh * (x - mean) * rstd, dbeta[H] = sum of dh (may be NULL).
 * ws: moe_layer_workspace_size bytes, 16-byte aligned. */
moe_status_t moe_layer_workspace_size(const moe_layer_t* cfg, size_t* bytes);
moe_status_t moe_layer_norm_backward(const moe_layer_t* cfg, const void* dh, const void* x,
                                     const float* gamma, const float* mean, const float* rstd,
                                     const void* dres, void* dx, float* dgamma, float* dbeta,
                                     void* ws, size_t ws_bytes, cudaStream_t stream);

/* out = x + scale * dropout(y), and with gamma_next the layer norm before the next block in the
 * same pass: h, mean, rstd of out as it is stored. gamma_next, h, mean and rstd are all given or
 * all NULL; beta_next may be NULL. out may be x or y. What is kept is rounded to fp32 as moe_dropout
 * stores it in fp32, then x is added. */
moe_status_t moe_dropout_join(const moe_layer_t* cfg, const moe_drop_t* drop, const void* x,
                              const void* y, const float* gamma_next, const float* beta_next,
                              void* out, void* h, float* mean, float* rstd, cudaStream_t stream);

/* Gradients of moe_dropout_join with a next norm, in one pass: d = dres + (gradient of the norm
 * from dh); dx = d, dy = scale * dropout(d), dgamma_next, dbeta_next (may be NULL). dres may be
 * NULL. (Without a next norm dx is dres, and dy is moe_dropout of it.) ws: as above. */
moe_status_t moe_dropout_join_backward(const moe_layer_t* cfg, const moe_drop_t* drop,
                                       const void* dres, const void* dh, const void* out,
                                       const float* gamma_next, const float* mean,
                                       const float* rstd, void* dx, void* dy, float* dgamma_next,
                                       float* dbeta_next, void* ws, size_t ws_bytes,
                                       cudaStream_t stream);

/* ---- balance and z losses of the router -----------------------------------------------
 * With z = logits (+ logit_bias, softmax routing only), p_te the softmax of a token's z (softmax
 * routing) or its sigmoids divided by their sum (sigmoid routing), and for sequence s with n_s
 * tokens that take part: counts[s, e] its slots whose id is e, P[s, e] the mean of p over its tokens:
 *
 *   balance = mean over sequences with n_s > 0 of  sum_e  E counts[s, e] / (k n_s) * P[s, e]
 *   z loss  = mean over tokens that take part of  (log sum_e exp z_te)^2
 *
 * both 0 where no token takes part. The gradient runs through P, not through the counts.
 * Sequence s is tokens offsets[s] <= t < offsets[s + 1]; tokens before the first or from the last
 * offset on, and tokens whose mask byte is 0, take no part, whatever their logits: their
 * dlogits are 0 (or, added to, left). Offsets do not decrease and lie in [0, T]; where they do not,
 * device status 5 is recorded (moe_device_status) and what the call writes is unspecified. Ids outside [0, E) and the n_shared
 * slots at the end are not counted. E at most 512, k + n_shared at most 32, T at most 2^28, S at most 2^20. */
typedef struct moe_balance {
  int T, E, k, n_shared;
  moe_route_mode_t mode;
  const float* logit_bias; /* fp32 [E] or NULL */
  int S;                   /* sequences; 1 without offsets */
  const int32_t* offsets;  /* device, [S + 1], or NULL: one sequence of all T tokens */
  const uint8_t* mask;     /* device, [T], or NULL */
} moe_balance_t;

/* losses[2] fp32 = {balance, z loss}, counts[S, E] int32, tokens[S] int32 = n_s, prob[S, E] fp32 = P
 * (0 where n_s = 0), totals[2] int32 = {sequences with n_s > 0, tokens that take part}. ws: 16-byte aligned. */
moe_status_t moe_balance_workspace_size(const moe_balance_t* cfg, size_t* bytes);
moe_status_t moe_balance_loss(const moe_balance_t* cfg, const float* logits, const int32_t* topk_ids,
                              float* losses, int32_t* counts, int32_t* tokens, float* prob,
                              int32_t* totals, void* ws, size_t ws_bytes, cudaStream_t stream);

/* dlogits[T, E] (+)= dlosses[0] d balance / d logits + dlosses[1] d z loss / d logits; dlosses[2]
 * fp32 on the device; counts, tokens, totals as moe_balance_loss wrote them. */
moe_status_t moe_balance_loss_backward(const moe_balance_t* cfg, const float* dlosses,
                                       const float* logits, const int32_t* counts,
                                       const int32_t* tokens, const int32_t* totals, int accumulate,
                                       float* dlogits, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_STACK_GB300_H */
