// route_grad.cu — gradient of the router weights with respect to the logits.
//
// With z = logits (+ logit_bias), C the chosen ids, g_e the gradient of the weight of e in C:
//   softmax over C (renormalised): p = softmax(z over C);  dz_e = scale p_e (g_e - sum_C g p)
//   softmax over all E:            p = softmax(z);         dz_e = scale p_e (g_e [e in C] - sum_C g p)
//   sigmoid, renormalised:         s = sigmoid(z), S = sum_C s, q = s / S:
//                                  dz_e = scale (g_e - sum_C g q) / S * s_e (1 - s_e)
//   sigmoid:                       dz_e = scale g_e s_e (1 - s_e)
// and zero for e outside C (but for the softmax over all E). Probabilities are computed from
// the logits again rather than divided back out of the stored weights. One warp a token, lane l
// holding experts l, l + 32, ...; the T*E writes (and, where the chosen ids alone matter,
// nothing but k logits of a row to read) bound it.
#include "train.cuh"

namespace moe {
namespace routeg {

constexpr int kWarps = 8;

template <int MPL>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, const float* __restrict__ bias, float* __restrict__ dlogits,
    int T, int E, int k, int slots, int mode, int renorm, float scale) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const float* row = logits + t * E;
  // lane j holds slot j; slots of ids outside [0, E) are left out
  int id = lane < k ? ids[t * slots + lane] : -1;
  if (id >= E) id = -1;
  const float g = id >= 0 ? dw[t * slots + lane] : 0.f;
  const bool dense = mode == MOE_ROUTE_SOFTMAX && !renorm;
  float z = id >= 0 ? row[id] : -INFINITY;
  if (id >= 0 && mode == MOE_ROUTE_SOFTMAX && bias) z += bias[id];

  float grad = 0.f;  // lane j: gradient of slot j's logit
  float p_all[MPL], dot = 0.f;
  if (dense) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < MPL; ++i) {
      const int e = lane + 32 * i;
      p_all[i] = -INFINITY;
      if (e < E) p_all[i] = bias ? row[e] + bias[e] : row[e];
      m = fmaxf(m, p_all[i]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < MPL; ++i) {
      p_all[i] = lane + 32 * i < E ? expf(p_all[i] - m) : 0.f;
      sum += p_all[i];
    }
    sum = warp_total(sum);
#pragma unroll
    for (int i = 0; i < MPL; ++i) p_all[i] /= sum;
    const float p = id >= 0 ? expf(z - m) / sum : 0.f;
    dot = warp_total(g * p);
    grad = scale * p * (g - dot);
  } else if (mode == MOE_ROUTE_SOFTMAX) {
    float m = z;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ex = id >= 0 ? expf(z - m) : 0.f;
    const float sum = warp_total(ex);
    const float p = id >= 0 ? ex / sum : 0.f;
    dot = warp_total(g * p);
    grad = scale * p * (g - dot);
  } else {
    // s and 1 - s each from the smaller exponential: taken from a rounded s, 1 - s would be off by
    // a thousandth of itself at z = 10 and zero from z = 17 on
    const float x = id >= 0 ? expf(-fabsf(z)) : 0.f;
    const float large = 1.f / (1.f + x), small = x * large;
    const float s = id >= 0 ? (z >= 0.f ? large : small) : 0.f, r = z >= 0.f ? small : large;
    float ds = g;
    if (renorm) {
      const float sum = warp_total(s);
      const float q = id >= 0 ? s / sum : 0.f;
      dot = warp_total(g * q);
      ds = id >= 0 ? (g - dot) / sum : 0.f;
    }
    grad = scale * ds * s * r;
  }

  float d[MPL];
#pragma unroll
  for (int i = 0; i < MPL; ++i) d[i] = dense ? -scale * p_all[i] * dot : 0.f;
  for (int j = 0; j < k; ++j) {
    const int ej = __shfl_sync(0xffffffffu, id, j);
    const float gj = __shfl_sync(0xffffffffu, grad, j);
    if (ej >= 0 && (ej & 31) == lane) {
#pragma unroll
      for (int i = 0; i < MPL; ++i)
        if (i == ej >> 5) d[i] = gj;
    }
  }
  float* out = dlogits + t * E;
#pragma unroll
  for (int i = 0; i < MPL; ++i)
    if (lane + 32 * i < E) out[lane + 32 * i] = d[i];
}

}  // namespace routeg

moe_status_t launch_route_backward(const moe_config_t& c, const float* logits,
                                   const int32_t* ids, const float* dw, float* dlogits,
                                   cudaStream_t s) {
  using namespace routeg;
  const dim3 grid((unsigned)ceil_div(c.T, kWarps)), block(kWarps * 32);
  auto go = [&](auto kern) {
    return launch_k(kern, grid, block, 0, s, logits, ids, dw,
                    c.mode == MOE_ROUTE_SOFTMAX ? c.logit_bias : (const float*)nullptr, dlogits,
                    c.T, c.E, c.k, c.k + c.n_shared, (int)c.mode, c.renormalize, c.scale);
  };
  if (c.E <= 128) return go(route_backward_kernel<4>);
  if (c.E <= 256) return go(route_backward_kernel<8>);
  return go(route_backward_kernel<16>);
}

}  // namespace moe
