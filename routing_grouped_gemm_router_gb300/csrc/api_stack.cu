// api_stack.cu — the C ABI of the operators around a stack's blocks (include/moe_stack.h): argument
// checks and which kernel takes a call. Nothing here allocates, synchronises or reads device memory.
#include <cmath>

#include "stack.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
bool dtype_ok(moe_dtype_t d) { return d == MOE_F32 || d == MOE_BF16; }

// All of the pointers given, on 16-byte boundaries; the same for words.
template <typename... P>
bool rows_ok(const P*... p) {
  return ((p != nullptr && aligned(p, 16)) && ...);
}
template <typename... P>
bool words_ok(const P*... p) {
  return ((p != nullptr && aligned(p, 4)) && ...);
}

moe_status_t check_layer(const moe_layer_t* c) {
  if (!c || c->T < 1 || c->H < 8 || c->H % 8 || !dtype_ok(c->dtype) || !(c->eps >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (c->H > 32768 || c->T > 1 << 30) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The dropout as the kernels take it, with the scale that goes into its factor.
moe_status_t make_drop(const moe_drop_t* d, float scale, Drop& out) {
  if (!d || !(d->p >= 0.0) || !(d->p < 1.0)) return MOE_ERR_INVALID_ARG;
  const double below = std::nearbyint(d->p * 4294967296.0);
  if (below >= 4294967296.0) return MOE_ERR_INVALID_ARG;  // nothing would be kept
  if (d->p > 0.0 && (!d->rng || !aligned(d->rng, 8))) return MOE_ERR_INVALID_ARG;
  out.rng = d->rng;
  out.below = (uint32_t)below;
  out.site = d->site;
  out.factor = (float)(scale / (1.0 - below / 4294967296.0));
  return MOE_OK;
}

moe_status_t check_embed(int T, int V, int H) {
  if (T < 1 || V < 1 || H < 8 || H % 8) return MOE_ERR_INVALID_ARG;
  if (T > 1 << 28 || V > 1 << 26 || H > 1 << 20) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
bool tokens_ok(const void* tokens, int token_bytes) {
  return tokens && (token_bytes == 4 || token_bytes == 8) && aligned(tokens, token_bytes);
}

moe_status_t check_balance(const moe_balance_t* c) {
  if (!c || c->T < 1 || c->E < 1 || c->k < 1 || c->k > c->E || c->n_shared < 0 || c->k > 32 ||
      c->n_shared > 32 - c->k || c->S < 1 || (!c->offsets && c->S != 1) ||
      (c->mode != MOE_ROUTE_SOFTMAX && c->mode != MOE_ROUTE_SIGMOID_GROUPED))
    return MOE_ERR_INVALID_ARG;
  if (c->E > 512 || c->T > 1 << 28 || c->S > 1 << 20) return MOE_ERR_UNSUPPORTED;
  if (!aligned(c->logit_bias, 4) || !aligned(c->offsets, 4)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_embed(const void* tokens, int token_bytes, int T, const void* table, int V, int H,
                       moe_dtype_t dtype, float scale, void* out, cudaStream_t stream) {
  const moe_status_t st = check_embed(T, V, H);
  if (st != MOE_OK) return st;
  if (!dtype_ok(dtype) || !tokens_ok(tokens, token_bytes) || !rows_ok(table, out))
    return MOE_ERR_INVALID_ARG;
  return launch_embed(tokens, token_bytes == 8, T, table, V, H, dtype, scale, out, stream);
}

moe_status_t moe_embed_workspace_size(int T, int V, int H, size_t* bytes) {
  const moe_status_t st = check_embed(T, V, H);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = embed_ws_bytes(T, V, H);
  return MOE_OK;
}

moe_status_t moe_embed_backward(const void* dx, const void* tokens, int token_bytes, int T, int V,
                                int H, moe_dtype_t dtype, moe_dtype_t out_dtype, float scale,
                                int accumulate, void* dtable, void* ws, size_t ws_bytes,
                                cudaStream_t stream) {
  const moe_status_t st = check_embed(T, V, H);
  if (st != MOE_OK) return st;
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype) || (dtype == MOE_F32 && out_dtype != MOE_F32) ||
      !tokens_ok(tokens, token_bytes) || !rows_ok(dx, dtable))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16) || ws_bytes < embed_ws_bytes(T, V, H)) return MOE_ERR_WORKSPACE;
  return launch_embed_backward(dx, tokens, token_bytes == 8, T, V, H, dtype, out_dtype, scale,
                               accumulate, dtable, ws, stream);
}

moe_status_t moe_dropout(const moe_layer_t* cfg, const moe_drop_t* drop, const void* x, void* out,
                         cudaStream_t stream) {
  moe_status_t st = check_layer(cfg);
  if (st != MOE_OK) return st;
  Drop d{};
  st = make_drop(drop, cfg->scale, d);
  if (st != MOE_OK) return st;
  if (!rows_ok(x, out)) return MOE_ERR_INVALID_ARG;
  return launch_dropout(*cfg, d, x, out, stream);
}

moe_status_t moe_layer_norm(const moe_layer_t* cfg, const void* x, const float* gamma,
                            const float* beta, void* h, float* mean, float* rstd,
                            cudaStream_t stream) {
  const moe_status_t st = check_layer(cfg);
  if (st != MOE_OK) return st;
  if (!rows_ok(x, gamma, h) || !aligned(beta, 16) || !words_ok(mean, rstd)) return MOE_ERR_INVALID_ARG;
  LayerArgs a{};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.h = h;
  a.mean = mean;
  a.rstd = rstd;
  return launch_layer_norm(*cfg, a, stream);
}

moe_status_t moe_layer_workspace_size(const moe_layer_t* cfg, size_t* bytes) {
  const moe_status_t st = check_layer(cfg);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = layer_ws_bytes(*cfg);
  return MOE_OK;
}

moe_status_t moe_layer_norm_backward(const moe_layer_t* cfg, const void* dh, const void* x,
                                     const float* gamma, const float* mean, const float* rstd,
                                     const void* dres, void* dx, float* dgamma, float* dbeta,
                                     void* ws, size_t ws_bytes, cudaStream_t stream) {
  const moe_status_t st = check_layer(cfg);
  if (st != MOE_OK) return st;
  if (!rows_ok(dh, x, gamma, dx) || !words_ok(mean, rstd, dgamma) || !aligned(dbeta, 4) ||
      !aligned(dres, 16))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16) || ws_bytes < layer_ws_bytes(*cfg)) return MOE_ERR_WORKSPACE;
  LayerArgs a{};
  a.dh = dh;
  a.x = x;
  a.gamma = gamma;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.dres = dres;
  a.dx = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.ws = (float*)ws;
  return launch_layer_norm_backward(*cfg, a, stream);
}

moe_status_t moe_dropout_join(const moe_layer_t* cfg, const moe_drop_t* drop, const void* x,
                              const void* y, const float* gamma_next, const float* beta_next,
                              void* out, void* h, float* mean, float* rstd, cudaStream_t stream) {
  moe_status_t st = check_layer(cfg);
  if (st != MOE_OK) return st;
  LayerArgs a{};
  st = make_drop(drop, cfg->scale, a.drop);
  if (st != MOE_OK) return st;
  if (!rows_ok(x, y, out)) return MOE_ERR_INVALID_ARG;
  if ((gamma_next || beta_next || h || mean || rstd) &&
      (!rows_ok(gamma_next, h) || !aligned(beta_next, 16) || !words_ok(mean, rstd)))
    return MOE_ERR_INVALID_ARG;
  a.x = x;
  a.y = y;
  a.gamma = gamma_next;
  a.beta = beta_next;
  a.out = out;
  a.h = h;
  a.mean = mean;
  a.rstd = rstd;
  return launch_dropout_join(*cfg, a, stream);
}

moe_status_t moe_dropout_join_backward(const moe_layer_t* cfg, const moe_drop_t* drop,
                                       const void* dres, const void* dh, const void* out,
                                       const float* gamma_next, const float* mean,
                                       const float* rstd, void* dx, void* dy, float* dgamma_next,
                                       float* dbeta_next, void* ws, size_t ws_bytes,
                                       cudaStream_t stream) {
  moe_status_t st = check_layer(cfg);
  if (st != MOE_OK) return st;
  LayerArgs a{};
  st = make_drop(drop, cfg->scale, a.drop);
  if (st != MOE_OK) return st;
  if (!rows_ok(dh, out, gamma_next, dx, dy) || !words_ok(mean, rstd, dgamma_next) ||
      !aligned(dbeta_next, 4) || !aligned(dres, 16))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16) || ws_bytes < layer_ws_bytes(*cfg)) return MOE_ERR_WORKSPACE;
  a.dres = dres;
  a.dh = dh;
  a.x = out;
  a.gamma = gamma_next;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.dx = dx;
  a.dy = dy;
  a.dgamma = dgamma_next;
  a.dbeta = dbeta_next;
  a.ws = (float*)ws;
  return launch_dropout_join_backward(*cfg, a, stream);
}

moe_status_t moe_balance_workspace_size(const moe_balance_t* cfg, size_t* bytes) {
  const moe_status_t st = check_balance(cfg);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = balance_ws_bytes(*cfg);
  return MOE_OK;
}

moe_status_t moe_balance_loss(const moe_balance_t* cfg, const float* logits, const int32_t* topk_ids,
                              float* losses, int32_t* counts, int32_t* tokens, float* prob,
                              int32_t* totals, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const moe_status_t st = check_balance(cfg);
  if (st != MOE_OK) return st;
  if (!words_ok(logits, topk_ids, losses, counts, tokens, prob, totals)) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 16) || ws_bytes < balance_ws_bytes(*cfg)) return MOE_ERR_WORKSPACE;
  return launch_balance(*cfg, logits, topk_ids, losses, counts, tokens, prob, totals, ws, stream);
}

moe_status_t moe_balance_loss_backward(const moe_balance_t* cfg, const float* dlosses,
                                       const float* logits, const int32_t* counts,
                                       const int32_t* tokens, const int32_t* totals, int accumulate,
                                       float* dlogits, cudaStream_t stream) {
  const moe_status_t st = check_balance(cfg);
  if (st != MOE_OK) return st;
  if (!words_ok(dlosses, logits, counts, tokens, totals, dlogits)) return MOE_ERR_INVALID_ARG;
  return launch_balance_backward(*cfg, dlosses, logits, counts, tokens, totals, accumulate, dlogits,
                                 stream);
}

}  // extern "C"
