// api_train.cu — the C ABI of the training operators (include/moe_train.h): argument checks
// and which kernel takes a call. Nothing here allocates, synchronises or reads device memory.
#include "train.cuh"

using namespace moe;

namespace {

// bf16 products run on the tensor cores, fp32 ones on the CUDA cores.
moe_status_t product(ExpertProduct kind, const moe_experts_t& c, const void* a, const void* w,
                     const float* h13, const int32_t* counts, void* out, void* act,
                     cudaStream_t s) {
  return c.dtype == MOE_BF16 ? launch_expert_product_tc(kind, c, a, w, h13, counts, out, act, s)
                             : launch_expert_product_simt(kind, c, a, w, h13, counts, out, act, s);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool dtype_ok(moe_dtype_t d) { return d == MOE_F32 || d == MOE_BF16; }

moe_status_t check_dispatch(int T, int k, int H, moe_dtype_t dt, int rows) {
  if (T < 1 || k < 1 || k > 32 || H < 8 || H % 8 || rows < 1 || !dtype_ok(dt))
    return MOE_ERR_INVALID_ARG;
  if ((int64_t)T * k > (int64_t)1 << 30 || rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t check_experts(const moe_experts_t* c) {
  if (!c || c->rows < 1 || c->E < 1 || c->H < 8 || c->I < 8 || c->H % 8 || c->I % 8 ||
      !dtype_ok(c->dtype))
    return MOE_ERR_INVALID_ARG;
  if (c->E > kMaxExperts || c->rows > kMaxRows || c->H > 1 << 20 || c->I > 1 << 20)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t check_block(const moe_block_t* c, bool join) {
  if (!c || c->T < 1 || c->H < 8 || c->H % 8 || !dtype_ok(c->dtype) || !(c->eps >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (join && (c->gate_kind < MOE_GATE_NONE || c->gate_kind > MOE_GATE_FULL))
    return MOE_ERR_INVALID_ARG;
  if (c->H > 32768 || c->T > 1 << 30) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// All of the pointers given, on 16-byte boundaries.
template <typename... P>
bool rows_ok(const P*... p) {
  return ((p != nullptr && aligned16(p)) && ...);
}
template <typename... P>
bool words_ok(const P*... p) {
  return ((p != nullptr && aligned4(p)) && ...);
}

}  // namespace

extern "C" {

moe_status_t moe_permute(const void* x, const int32_t* topk_ids, const int32_t* sorted_ids,
                         int T, int k, int E, int H, moe_dtype_t dtype, int rows, void* xs,
                         int32_t* row_pos, cudaStream_t stream) {
  const moe_status_t st = check_dispatch(T, k, H, dtype, rows);
  if (st != MOE_OK) return st;
  if (E < 1 || !rows_ok(x, xs) || !words_ok(topk_ids, sorted_ids, row_pos))
    return MOE_ERR_INVALID_ARG;
  return launch_permute(x, topk_ids, sorted_ids, T, k, E, H, dtype, rows, xs, row_pos, stream);
}

moe_status_t moe_permute_backward(const void* dxs, const int32_t* row_pos, int T, int k, int H,
                                  moe_dtype_t dtype, int rows, void* dx, cudaStream_t stream) {
  const moe_status_t st = check_dispatch(T, k, H, dtype, rows);
  if (st != MOE_OK) return st;
  if (!rows_ok(dxs, dx) || !words_ok(row_pos)) return MOE_ERR_INVALID_ARG;
  return launch_slot_sum(dxs, row_pos, nullptr, T, k, H, dtype, rows, dx, stream);
}

moe_status_t moe_unpermute(const void* ys, const int32_t* row_pos, const float* topk_w, int T,
                           int k, int H, moe_dtype_t dtype, int rows, void* out,
                           cudaStream_t stream) {
  const moe_status_t st = check_dispatch(T, k, H, dtype, rows);
  if (st != MOE_OK) return st;
  if (!rows_ok(ys, out) || !words_ok(row_pos, topk_w)) return MOE_ERR_INVALID_ARG;
  return launch_slot_sum(ys, row_pos, topk_w, T, k, H, dtype, rows, out, stream);
}

moe_status_t moe_unpermute_backward(const void* dout, const void* ys, const int32_t* sorted_ids,
                                    const int32_t* row_pos, const float* topk_w, int T, int k,
                                    int H, moe_dtype_t dtype, int rows, void* dys,
                                    float* dtopk_w, cudaStream_t stream) {
  const moe_status_t st = check_dispatch(T, k, H, dtype, rows);
  if (st != MOE_OK) return st;
  if (!rows_ok(dout, ys, dys) || !words_ok(sorted_ids, row_pos, topk_w, dtopk_w))
    return MOE_ERR_INVALID_ARG;
  return launch_unpermute_backward(dout, ys, sorted_ids, row_pos, topk_w, T, k, H, dtype, rows,
                                   dys, dtopk_w, stream);
}

moe_status_t moe_expert_up(const moe_experts_t* cfg, const void* xs, const void* W13,
                           const int32_t* counts, float* h13, void* act, cudaStream_t stream) {
  const moe_status_t st = check_experts(cfg);
  if (st != MOE_OK) return st;
  if (!rows_ok(xs, W13, h13, act) || !words_ok(counts)) return MOE_ERR_INVALID_ARG;
  return product(kUp, *cfg, xs, W13, nullptr, counts, h13, act, stream);
}

moe_status_t moe_expert_down(const moe_experts_t* cfg, const void* act, const void* W2,
                             const int32_t* counts, void* ys, cudaStream_t stream) {
  const moe_status_t st = check_experts(cfg);
  if (st != MOE_OK) return st;
  if (!rows_ok(act, W2, ys) || !words_ok(counts)) return MOE_ERR_INVALID_ARG;
  return product(kDown, *cfg, act, W2, nullptr, counts, ys, nullptr, stream);
}

moe_status_t moe_expert_down_backward(const moe_experts_t* cfg, const void* dys, const void* W2,
                                      const float* h13, const int32_t* counts, void* dh13,
                                      void* act, cudaStream_t stream) {
  const moe_status_t st = check_experts(cfg);
  if (st != MOE_OK) return st;
  if (!rows_ok(dys, W2, h13, dh13, act) || !words_ok(counts)) return MOE_ERR_INVALID_ARG;
  return product(kDownGrad, *cfg, dys, W2, h13, counts, dh13, act, stream);
}

moe_status_t moe_expert_up_backward(const moe_experts_t* cfg, const void* dh13, const void* W13,
                                    const int32_t* counts, void* dxs, cudaStream_t stream) {
  const moe_status_t st = check_experts(cfg);
  if (st != MOE_OK) return st;
  if (!rows_ok(dh13, W13, dxs) || !words_ok(counts)) return MOE_ERR_INVALID_ARG;
  return product(kUpGrad, *cfg, dh13, W13, nullptr, counts, dxs, nullptr, stream);
}

moe_status_t moe_expert_weight_grad(int rows, int E, int M, int N, moe_dtype_t dtype,
                                    moe_dtype_t out_dtype, int accumulate, const void* dy,
                                    const void* a, const int32_t* counts, void* dW,
                                    cudaStream_t stream) {
  if (rows < 1 || E < 1 || M < 8 || N < 8 || M % 8 || N % 8 || !dtype_ok(dtype) ||
      !dtype_ok(out_dtype) || (dtype == MOE_F32 && out_dtype != MOE_F32))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || rows > kMaxRows || M > 1 << 21 || N > 1 << 21) return MOE_ERR_UNSUPPORTED;
  if (!rows_ok(dy, a, dW) || !words_ok(counts)) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_BF16)
    return launch_weight_grad_tc(rows, E, M, N, out_dtype, accumulate, dy, a, counts, dW, stream);
  return launch_weight_grad_simt(rows, E, M, N, accumulate, dy, a, counts, dW, stream);
}

moe_status_t moe_block_workspace_size(const moe_block_t* cfg, size_t* bytes) {
  const moe_status_t st = check_block(cfg, true);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = block_norm_ws_bytes(*cfg);
  return MOE_OK;
}

moe_status_t moe_block_norm(const moe_block_t* cfg, const void* x, const float* gamma, void* h,
                            float* rstd, cudaStream_t stream) {
  const moe_status_t st = check_block(cfg, false);
  if (st != MOE_OK) return st;
  if (!rows_ok(x, gamma, h) || !words_ok(rstd)) return MOE_ERR_INVALID_ARG;
  BlockNormArgs a{};
  a.x = x;
  a.gamma = gamma;
  a.h = h;
  a.rstd_out = rstd;
  return launch_block_norm(*cfg, a, stream);
}

moe_status_t moe_block_norm_backward(const moe_block_t* cfg, const void* dh, const void* x,
                                     const float* gamma, const float* rstd, const void* dres,
                                     void* dx, float* dgamma, void* ws, size_t ws_bytes,
                                     cudaStream_t stream) {
  const moe_status_t st = check_block(cfg, false);
  if (st != MOE_OK) return st;
  if (!rows_ok(dh, x, gamma, dx) || !words_ok(rstd, dgamma) || !aligned16(dres))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < block_norm_ws_bytes(*cfg)) return MOE_ERR_WORKSPACE;
  BlockNormArgs a{};
  a.dh = dh;
  a.x = x;
  a.gamma = gamma;
  a.rstd_y_in = rstd;
  a.dres = dres;
  a.dx = dx;
  a.dgamma = dgamma;
  a.ws = (float*)ws;
  return launch_block_norm_backward(*cfg, a, stream);
}

moe_status_t moe_block_join(const moe_block_t* cfg, const void* x, const void* y,
                            const float* gamma, const void* gate, const float* gamma_next,
                            void* out, float* rstd_y, void* h, float* rstd_out,
                            cudaStream_t stream) {
  const moe_status_t st = check_block(cfg, true);
  if (st != MOE_OK) return st;
  if (!rows_ok(x, y, gamma, out) || !words_ok(rstd_y) || !aligned16(gate))
    return MOE_ERR_INVALID_ARG;
  if ((cfg->gate_kind != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((gamma_next || h || rstd_out) && (!rows_ok(gamma_next, h) || !words_ok(rstd_out)))
    return MOE_ERR_INVALID_ARG;
  BlockNormArgs a{};
  a.x = x;
  a.y = y;
  a.gamma = gamma;
  a.gate = gate;
  a.gamma_next = gamma_next;
  a.out = out;
  a.rstd_y = rstd_y;
  a.h = h;
  a.rstd_out = rstd_out;
  return launch_block_join(*cfg, a, stream);
}

moe_status_t moe_block_join_backward(const moe_block_t* cfg, const void* dres, const void* dh,
                                     const void* out, const void* y, const float* gamma,
                                     const void* gate, const float* gamma_next,
                                     const float* rstd_y, const float* rstd_out, void* dx,
                                     void* dy, float* dgamma, float* dgamma_next, void* dgate,
                                     void* ws, size_t ws_bytes, cudaStream_t stream) {
  const moe_status_t st = check_block(cfg, true);
  if (st != MOE_OK) return st;
  if (!rows_ok(y, gamma, dx, dy) || !words_ok(rstd_y, dgamma) || !aligned16(gate) ||
      !aligned16(dgate) || !aligned16(dres))
    return MOE_ERR_INVALID_ARG;
  if ((cfg->gate_kind != MOE_GATE_NONE) != (gate != nullptr) || !gate != !dgate)
    return MOE_ERR_INVALID_ARG;
  if ((dh || out || gamma_next || rstd_out || dgamma_next) &&
      (!rows_ok(dh, out, gamma_next) || !words_ok(rstd_out, dgamma_next)))
    return MOE_ERR_INVALID_ARG;
  if (!gamma_next && !dres) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < block_norm_ws_bytes(*cfg)) return MOE_ERR_WORKSPACE;
  BlockNormArgs a{};
  a.dres = dres;
  a.dh = dh;
  a.out_in = out;
  a.y = y;
  a.gamma = gamma;
  a.gate = gate;
  a.gamma_next = gamma_next;
  a.rstd_y_in = rstd_y;
  a.rstd_out_in = rstd_out;
  a.dx = dx;
  a.dy = dy;
  a.dgamma = dgamma;
  a.dgamma_next = dgamma_next;
  a.dgate = dgate;
  a.ws = (float*)ws;
  return launch_block_join_backward(*cfg, a, stream);
}

moe_status_t moe_route_backward(const moe_config_t* cfg, const float* logits,
                                const int32_t* topk_ids, const float* dtopk_w, float* dlogits,
                                cudaStream_t stream) {
  if (!cfg || cfg->T < 1 || cfg->E < 1 || cfg->k < 1 || cfg->k > cfg->E || cfg->k > 32 ||
      cfg->n_shared < 0 || cfg->n_shared > 8 || cfg->k + cfg->n_shared > 32 ||
      (cfg->mode != MOE_ROUTE_SOFTMAX && cfg->mode != MOE_ROUTE_SIGMOID_GROUPED))
    return MOE_ERR_INVALID_ARG;
  if (cfg->E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  if (!words_ok(logits, topk_ids, dtopk_w, dlogits) || !aligned4(cfg->logit_bias))
    return MOE_ERR_INVALID_ARG;
  return launch_route_backward(*cfg, logits, topk_ids, dtopk_w, dlogits, stream);
}

}  // extern "C"
