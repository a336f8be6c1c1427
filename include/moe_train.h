/*
 * moe_train.h — C ABI of the operators that train a sparse block on GB300 (sm_103a): the
 * dispatch of token rows to experts and back with its gradients, the experts' grouped
 * products with theirs, the norms before and after the block fused with its gate and
 * residual scale, and the router's gradient. Same library, statuses and conventions as
 * moe.h: device pointers, contiguous row-major tensors, 16-byte aligned rows, the caller owns
 * every buffer, nothing allocates, synchronises or reads device data on the host, argument
 * errors come back before anything is enqueued, every call can be captured in a CUDA graph.
 *
 * One training step of the block (n = T*k routed slots, slot r = t*k + j):
 *
 *   h        = moe_block_norm(x)                              norm before the block
 *   logits, topk_ids, topk_w = moe_route(h)                   (moe.h)
 *   sorted_ids, counts       = moe_align(topk_ids, block 16)  (moe.h)
 *   xs, row_pos = moe_permute(h)                              rows of one expert together
 *   h13, act = moe_expert_up(xs);  ys = moe_expert_down(act)
 *   y        = moe_unpermute(ys, topk_w)
 *   out      = moe_block_join(x, y)                           x + scale * gate . norm(y)
 *
 * and backwards, in the opposite order, through the *_backward calls.
 *
 * Row layout. Expert e's rows are counts[e] consecutive rows of a P-row buffer, starting at
 * the sum over lower experts of their counts rounded up to MOE_TRAIN_BLOCK rows: the table
 * that moe_align writes for block_m = MOE_TRAIN_BLOCK, with
 * P = moe_max_padded_rows(T, k, E, MOE_TRAIN_BLOCK). Sixteen rows are one K step of the
 * tensor cores' bf16 MMA, so the weight gradients' reduction over an expert's rows wastes at
 * most one step. Rows that hold no slot (padding, and the tail up to P) are written as zeros
 * by every call that writes such a buffer, and the expert products need them to be zero in
 * what they read. Counts that do not fit in P rows (or are negative) are cut, and device
 * status 4 is recorded (moe_device_status).
 */
#ifndef MOE_TRAIN_GB300_H
#define MOE_TRAIN_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_TRAIN_BLOCK 16 /* rows an expert's run is padded to */

/* ---- dispatch -------------------------------------------------------------------------
 * T >= 1 tokens, 1 <= k <= 32 slots each, H a multiple of 8, rows = P >= 1 buffer rows.
 * row_pos[T, k] int32 is the row of each slot, -1 for a slot whose expert id lies outside
 * [0, E) (dropped: it adds nothing and gets no gradient). Entries of row_pos outside
 * [0, rows) count as dropped, entries of sorted_ids outside [0, T*k) as rows of no slot. */

/* xs[p] = x[sorted_ids[p] / k] (zeros in rows of no slot, for all rows p < rows) and
 * row_pos[sorted_ids[p]] = p. */
moe_status_t moe_permute(const void* x, const int32_t* topk_ids, const int32_t* sorted_ids,
                         int T, int k, int E, int H, moe_dtype_t dtype, int rows, void* xs,
                         int32_t* row_pos, cudaStream_t stream);

/* dx[t] = sum_j dxs[row_pos[t, j]], summed in fp32 in slot order. */
moe_status_t moe_permute_backward(const void* dxs, const int32_t* row_pos, int T, int k, int H,
                                  moe_dtype_t dtype, int rows, void* dx, cudaStream_t stream);

/* out[t] = sum_j topk_w[t, j] * ys[row_pos[t, j]], summed in fp32 in slot order. */
moe_status_t moe_unpermute(const void* ys, const int32_t* row_pos, const float* topk_w, int T,
                           int k, int H, moe_dtype_t dtype, int rows, void* out,
                           cudaStream_t stream);

/* dys[row_pos[t, j]] = topk_w[t, j] * dout[t] (zeros in rows of no slot) and
 * dtopk_w[t, j] = <dout[t], ys[row_pos[t, j]]> in fp32 (0 for dropped slots). */
moe_status_t moe_unpermute_backward(const void* dout, const void* ys, const int32_t* sorted_ids,
                                    const int32_t* row_pos, const float* topk_w, int T, int k,
                                    int H, moe_dtype_t dtype, int rows, void* dys,
                                    float* dtopk_w, cudaStream_t stream);

/* ---- experts --------------------------------------------------------------------------
 * W13[E, 2I, H] (gate rows 0..I-1, up rows I..2I-1), W2[E, H, I], row buffers of `rows` rows in
 * the layout above, all in dtype; counts[E] int32 on the device. H and I multiples of 8,
 * E <= 512. bf16 products run on the tensor cores with fp32 accumulation, fp32 ones on the
 * CUDA cores. */
typedef struct moe_experts {
  int rows; /* P: rows of every row buffer */
  int E, H, I;
  moe_dtype_t dtype;
} moe_experts_t;

/* h13[rows, 2I] = xs W13[e]^T (gate, then up) in fp32 for either dtype, kept for the backward
 * pass, whose gradients then carry no rounding but that of dh13 and act: with bf16 kept instead,
 * the gradients of W13 measured twice the error of a single rounding, with fp32 1.4 times. And
 * act[rows, I] = silu(gate) * up, from the fp32 sums. */
moe_status_t moe_expert_up(const moe_experts_t* cfg, const void* xs, const void* W13,
                           const int32_t* counts, float* h13, void* act, cudaStream_t stream);

/* ys[rows, H] = act W2[e]^T. */
moe_status_t moe_expert_down(const moe_experts_t* cfg, const void* act, const void* W2,
                             const int32_t* counts, void* ys, cudaStream_t stream);

/* Gradient through W2 and the SwiGLU: with dact = dys W2[e] (fp32, never stored), s = sigmoid(gate):
 *   dh13[:, :I] = dact * up * s * (1 + gate * (1 - s)),  dh13[:, I:] = dact * gate * s,
 *   act = silu(gate) * up, recomputed from h13 for the gradient of W2, so that the forward
 * pass need not keep it. */
moe_status_t moe_expert_down_backward(const moe_experts_t* cfg, const void* dys, const void* W2,
                                      const float* h13, const int32_t* counts, void* dh13,
                                      void* act, cudaStream_t stream);

/* dxs[rows, H] = dh13 W13[e]. */
moe_status_t moe_expert_up_backward(const moe_experts_t* cfg, const void* dh13, const void* W13,
                                    const int32_t* counts, void* dxs, cudaStream_t stream);

/* dW[e] (+)= dy_e^T a_e over expert e's rows: dy[rows, M], a[rows, N], dW[E, M, N].
 * W2's gradient takes dy = dys, a = act (M = H, N = I), W13's dy = dh13, a = xs (M = 2I,
 * N = H). dtype is that of dy and a; out_dtype (MOE_F32, or MOE_BF16 when dtype is) that of
 * dW. accumulate 0: dW is overwritten (zeros for an expert without rows); 1: added to, the sum
 * rounded once. The tensor cores' accumulators cut off rather than round; fp32 dW of bf16 rows leaves them
 * every 512 rows and is added up in rounded fp32 (off by 4.8e-7 of its size over 512 to 8192 rows). fp32
 * products and their gradients sum in fp32, reductions of more than 2048 steps in spans of 512. */
moe_status_t moe_expert_weight_grad(int rows, int E, int M, int N, moe_dtype_t dtype,
                                    moe_dtype_t out_dtype, int accumulate, const void* dy,
                                    const void* a, const int32_t* counts, void* dW,
                                    cudaStream_t stream);

/* ---- norms around the block -----------------------------------------------------------
 * Rows of H elements (a multiple of 8, at most 32768). Norm weights, per-channel and per-token
 * gates and all their gradients are fp32; rows are dtype. The weight used is
 * offset + gamma (offset 1 for weights kept as a difference from one). rstd is
 * 1 / sqrt(mean of squares + eps), fp32 [T], kept for the backward pass. */
typedef enum {
  MOE_GATE_NONE = 0,
  MOE_GATE_CHANNEL = 1, /* fp32 [H], shared by all tokens */
  MOE_GATE_TOKEN = 2,   /* fp32 [T], shared by a token's channels */
  MOE_GATE_FULL = 3     /* dtype [T, H] */
} moe_gate_t;

typedef struct moe_block {
  int T, H;
  moe_dtype_t dtype;
  moe_gate_t gate_kind; /* join calls */
  float scale;          /* join calls: residual scale */
  float offset;
  float eps;
} moe_block_t;

/* h = x * rstd * (offset + gamma). */
moe_status_t moe_block_norm(const moe_block_t* cfg, const void* x, const float* gamma, void* h,
                            float* rstd, cudaStream_t stream);

/* dx = dres + d norm / dx (dres, the gradient that reaches x past the norm, may be NULL) and
 * dgamma[H] = sum over tokens of dh * x * rstd. ws: moe_block_workspace_size bytes, 16-byte aligned. */
moe_status_t moe_block_workspace_size(const moe_block_t* cfg, size_t* bytes);
moe_status_t moe_block_norm_backward(const moe_block_t* cfg, const void* dh, const void* x,
                                     const float* gamma, const float* rstd, const void* dres,
                                     void* dx, float* dgamma, void* ws, size_t ws_bytes,
                                     cudaStream_t stream);

/* out = x + scale * gate * (y * rstd_y * (offset + gamma)), and with gamma_next the norm before
 * the next block of the same pass: h = out * rstd_out * (offset + gamma_next), read from out as
 * it is stored. Both norms have cfg's eps and offset; a next norm with others is a moe_block_norm
 * of out, and moe_block_join_backward takes its rstd as rstd_out. gamma_next, h and rstd_out are
 * all given or all NULL. out may be x. */
moe_status_t moe_block_join(const moe_block_t* cfg, const void* x, const void* y,
                            const float* gamma, const void* gate, const float* gamma_next,
                            void* out, float* rstd_y, void* h, float* rstd_out,
                            cudaStream_t stream);

/* Gradients of moe_block_join in one pass: d = dres + (gradient of the next norm from dh), then
 *   dx = d, dy, dgamma, dgamma_next, dgate (shape and type of the gate; gradients of shared
 * gates are summed over what shares them, in a fixed order).
 * dres: gradient that reaches out past the next norm, or NULL (0). dh, out, gamma_next,
 * rstd_out, dgamma_next: all given or all NULL (no next norm; dres then has to be given). dgate
 * is NULL exactly when gate is. ws: moe_block_workspace_size bytes, 16-byte aligned. */
moe_status_t moe_block_join_backward(const moe_block_t* cfg, const void* dres, const void* dh,
                                     const void* out, const void* y, const float* gamma,
                                     const void* gate, const float* gamma_next,
                                     const float* rstd_y, const float* rstd_out, void* dx,
                                     void* dy, float* dgamma, float* dgamma_next, void* dgate,
                                     void* ws, size_t ws_bytes, cudaStream_t stream);

/* ---- router ---------------------------------------------------------------------------
 * dlogits[T, E] fp32 from the gradient of the router weights, dtopk_w[T, k + n_shared] fp32:
 * the derivative of moe_route's topk_w with respect to its logits, for the ids it chose
 * (the choice itself has no gradient; shared experts' slots and ids outside [0, E) are
 * skipped). Every entry is written: zeros outside the chosen ids, except in softmax mode
 * without renormalisation, where every probability depends on every logit. cfg as for
 * moe_route (H, I and the weights' fields are ignored). */
moe_status_t moe_route_backward(const moe_config_t* cfg, const float* logits,
                                const int32_t* topk_ids, const float* dtopk_w, float* dlogits,
                                cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_TRAIN_GB300_H */
