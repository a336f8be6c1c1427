// layer_norm.cu — the layer norm, the residual join with dropout that takes the next layer norm in
// the same pass, and their gradients (moe_layer_norm, moe_dropout_join and their backward calls).
//
// With m = mean(x), r = (mean((x - m)^2) + eps)^-1/2, xn = (x - m) r, keep the mask over 1 - p:
//   norm   h = xn gamma + beta
//   join   out = x + scale keep y;  h = norm(out)
//   back   a = dh gamma:  d = dres + r (a - mean(a) - xn mean(a xn));  dx = d,  dy = scale keep d
//          dgamma = sum_t dh xn;  dbeta = sum_t dh
// Every row is read once and written once, so HBM bounds all of them: rows go through the rings and
// the column sums of row_ring.cuh. The mask is computed from the element's number wherever it is needed.
//
// The variance is summed about a mean that is already near the row's: a warp sums its own elements,
// then their squared distances from its own mean, and the warps' sums and distances are joined by
//   M2 = sum_w M2_w + n_w (m_w - m)^2.
// That takes two rounds of shuffles and one barrier a row, where a mean first and the squares after
// take two, and it loses nothing for rows whose mean is large against their spread, where a
// difference of squares would.
#include "row_ring.cuh"
#include "stack.cuh"

namespace moe {
namespace lnorm {

using namespace rows;

// ------------------------------------------------------------------- forward
// Elements that warp `w` of a row's group holds.
template <int VPT>
__device__ __forceinline__ float warp_elements(const Shape& S, int w) {
  int n = 0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) n += min(max(S.chunks - (w * 32 + v * S.group), 0), 32);
  return 8.f * n;
}

// Keeps or drops eight elements and scales them: y * factor, or 0 whatever y is.
template <bool DROP>
__device__ __forceinline__ void drop_scale(F2 (&y)[4], const Philox* rng, const Drop& d,
                                           int64_t first) {
  if (DROP) {
    uint32_t w[8];
    rng->eight(first, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      split(y[i], lo, hi);
      y[i] = f2(w[2 * i] >= d.below ? lo : 0.f, w[2 * i + 1] >= d.below ? hi : 0.f) * dup(d.factor);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = y[i] * dup(d.factor);
  }
}

// JOIN: out = x + scale dropout(y), then (if gamma) its norm; otherwise the norm of x. Row tensors: JOIN y,
// x; otherwise x.
template <typename T, int VPT, int THREADS, bool JOIN, bool DROP>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 4 / VPT + 1 : 1)
    forward_kernel(const __grid_constant__ Shape S, const __grid_constant__ LayerArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Reducer red;
  const int local = threadIdx.x / S.group, g = threadIdx.x - local * S.group;
  const int lane = threadIdx.x & 31, warps = S.group >> 5;
  Ring<T, VPT, 2> ring(S, smem, local, g);
  const float inv_mine = 1.f / fmaxf(warp_elements<VPT>(S, g >> 5), 1.f);
  const float n_lane = lane < warps ? warp_elements<VPT>(S, lane) : 0.f;
  const float inv_lane = 1.f / fmaxf(n_lane, 1.f);
  pdl_wait();
  pdl_trigger();
  ring.start();
  Philox rng = DROP ? Philox(A.drop) : Philox();
  int turn = 0;
  for (int u = blockIdx.x; u < S.units; u += gridDim.x) {
    const int t = u * S.per + local;
    const bool live = t < S.T;
    const int tl = live ? t : 0;
    const int64_t row = (int64_t)tl * S.H;
    ring.wait();
    F2 o[VPT][4], s = dup(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!ring.has[v] || !live) continue;
      Chunk<T> q;
      ring.get(q, 0, v, tl);
      q.get(o[v]);
      if (JOIN) {
        drop_scale<DROP>(o[v], &rng, A.drop, row + c * 8);
        Chunk<T> xq;
        F2 x[4];
        ring.get(xq, 1, v, tl);
        xq.get(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[v][i] = o[v][i] + x[i];
        q.set(o[v]);
        q.store(A.out, row + c * 8);
        q.get(o[v]);  // the norm reads what is stored
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s = s + o[v][i];
    }
    const float sum = warp_total(both(s));
    ring.refill(u);
    if (JOIN && !A.gamma) continue;
    const F2 near = dup(-sum * inv_mine);
    s = dup(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (!ring.has[v] || !live) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 d = o[v][i] + near;
        s = fma2(d, d, s);
      }
    }
    float m2 = warp_total(both(s)), mean = sum * S.inv_h;
    if (warps > 1) {
      auto& buf = red.buf[turn];
      turn ^= 1;
      const int w = threadIdx.x >> 5, first = w - (g >> 5);
      if (lane == 0) {
        buf[0][w] = sum;
        buf[1][w] = m2;
      }
      __syncthreads();
      const float sw = lane < warps ? buf[0][first + lane] : 0.f;
      mean = warp_total(sw) * S.inv_h;
      const float off = sw * inv_lane - mean;
      m2 = warp_total(lane < warps ? fmaf(n_lane * off, off, buf[1][first + lane]) : 0.f);
    }
    if (!live) continue;
    const float r = rsqrtf(m2 * S.inv_h + S.eps);
    if (g == 0) {
      A.mean[t] = mean;
      A.rstd[t] = r;
    }
    const F2 rr = dup(r), mm = dup(-mean);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!ring.has[v]) continue;
      F2 ga[4], be[4];
      load_w(A.gamma, c * 8, ga);
      if (A.beta) load_w(A.beta, c * 8, be);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 xn = (o[v][i] + mm) * rr;
        ga[i] = A.beta ? fma2(xn, ga[i], be[i]) : xn * ga[i];
      }
      Chunk<T> q;
      q.set(ga);
      q.store(A.h, row + c * 8);
    }
  }
}

// ------------------------------------------------------------------- backward
// JOIN: dy too. RES: dres is there. Row tensors: dh, x, (dres).
template <typename T, int VPT, int THREADS, bool JOIN, bool DROP, bool RES>
__global__ void __launch_bounds__(THREADS, VPT <= 2 && THREADS <= 256 ? 2 : 1)
    backward_kernel(const __grid_constant__ Shape S, const __grid_constant__ LayerArgs A, int kinds,
                    const Outs outs) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Reducer red;
  const int local = threadIdx.x / S.group, g = threadIdx.x - local * S.group;
  Ring<T, VPT, 3> ring(S, smem, local, g);
  pdl_wait();
  pdl_trigger();
  ring.start();
  Philox rng = DROP ? Philox(A.drop) : Philox();
  int turn = 0;
  const F2 zero = dup(0.f);
  F2 sg[VPT][4], sb[VPT][4];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) sg[v][i] = sb[v][i] = zero;

  // a row's scalars are asked for one row ahead: nothing else hides their way from L2
  float m_next = 0.f, r_next = 0.f;
  auto scalars = [&](int64_t t) {
    if (t >= S.T) t = 0;
    m_next = __ldg(A.mean_in + t);
    r_next = __ldg(A.rstd_in + t);
  };
  scalars((int64_t)blockIdx.x * S.per + local);
  for (int u = blockIdx.x; u < S.units; u += gridDim.x) {
    const int t = u * S.per + local;
    const bool live = t < S.T;
    const int tl = live ? t : 0;
    const int64_t row = (int64_t)tl * S.H;
    const float r = r_next;
    const F2 rr = dup(r), shift = dup(-m_next * r);  // xn = x r + shift
    const F2 mm = dup(-m_next);
    scalars((int64_t)t + (int64_t)gridDim.x * S.per);
    ring.wait();
    Chunk<T> xq[VPT];
    F2 d[VPT][4], s1 = zero, s2 = zero;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!ring.has[v] || !live) continue;
      Chunk<T> q;
      F2 x[4], ga[4];
      ring.get(q, 0, v, tl);
      ring.get(xq[v], 1, v, tl);
      q.get(d[v]);
      xq[v].get(x);
      load_w(A.gamma, c * 8, ga);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 xn = (x[i] + mm) * rr;
        sg[v][i] = fma2(d[v][i], xn, sg[v][i]);
        sb[v][i] = sb[v][i] + d[v][i];
        d[v][i] = d[v][i] * ga[i];
        s1 = fma2(d[v][i], xn, s1);
        s2 = s2 + d[v][i];
      }
      if (RES) {
        F2 f[4];
        ring.get(q, 2, v, tl);
        q.get(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] = fma2(d[v][i], rr, f[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] = d[v][i] * rr;
      }
    }
    float s[2] = {both(s1), both(s2)};
    group_sum<2>(s, S.group, red, turn);
    ring.refill(u);
    // dx = d - r mean(a) - r mean(a xn) xn
    const F2 m1 = dup(-s[0] * S.inv_h * r), m0 = dup(-s[1] * S.inv_h * r);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!ring.has[v] || !live) continue;
      F2 x[4];
      xq[v].get(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[v][i] = fma2((x[i] + mm) * rr, m1, d[v][i] + m0);
      Chunk<T> o;
      o.set(d[v]);
      o.store(A.dx, row + c * 8);
      if (JOIN) {
        drop_scale<DROP>(d[v], &rng, A.drop, row + c * 8);
        o.set(d[v]);
        o.store(A.dy, row + c * 8);
      }
    }
  }
  leave_columns<VPT>(S, smem, local, g, sg, 0, kinds, 1.f, A.ws, outs);
  if (kinds > 1) leave_columns<VPT>(S, smem, local, g, sb, 1, kinds, 1.f, A.ws, outs);
}

// Chunks of 8 elements a thread holds: as many as it takes for a row to have at most 256 threads (bf16,
// up to 8192 channels) or 448 (fp32, up to 7168, where more chunks would not fit the ring), and twice as
// many threads or chunks beyond. The backward kernels hold 24 registers of sums and gradients a chunk, so
// a row's threads are capped where the chunks are counted.
static int vec_of(const moe_layer_t& c) {
  const int chunks = c.H / 8;
  if (c.dtype == MOE_F32) return chunks <= 32 ? 1 : chunks <= 896 ? 2 : chunks <= 2048 ? 4 : 8;
  return chunks <= 32 ? 1 : chunks <= 512 ? 2 : chunks <= 2048 ? 4 : 8;
}
static Shape shape_of(const moe_layer_t& c) {
  Shape s{};
  s.T = c.T;
  s.H = c.H;
  s.chunks = c.H / 8;
  s.group = ceil_div(ceil_div(s.chunks, vec_of(c)), 32) * 32;
  s.per = std::min(c.T, std::max(1, 256 / s.group));
  s.units = ceil_div(c.T, s.per);
  s.scale = c.scale;
  s.eps = c.eps;
  s.inv_h = 1.0f / (float)c.H;
  return s;
}

using bf = __nv_bfloat16;

// The kernel instance of a dtype and a row length.
#define LNORM_PICK(name, ...)                                                                 \
  (c.dtype == MOE_BF16 ? (v == 1   ? go(name<bf, 1, 256, __VA_ARGS__>)                        \
                          : v == 2 ? go(name<bf, 2, 256, __VA_ARGS__>)                        \
                          : v == 4 ? (c.H <= 8192 ? go(name<bf, 4, 256, __VA_ARGS__>)         \
                                                  : go(name<bf, 4, 512, __VA_ARGS__>))        \
                                   : go(name<bf, 8, 512, __VA_ARGS__>))                       \
                       : (v == 1   ? go(name<float, 1, 256, __VA_ARGS__>)                     \
                          : v == 2 ? go(name<float, 2, 448, __VA_ARGS__>)                     \
                          : v == 4 ? go(name<float, 4, 512, __VA_ARGS__>)                     \
                                   : go(name<float, 8, 512, __VA_ARGS__>)))

template <bool JOIN, bool DROP>
static moe_status_t forward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  Shape S = shape_of(c);
  if (JOIN) S.in[S.n_in++] = a.y;
  S.in[S.n_in++] = a.x;
  int blocks = 0;
  const int v = vec_of(c);
  auto go = [&](auto kern) {
    return run(kern, S, dtype_size(c.dtype), 0, v * dtype_size(c.dtype) <= 8, 8, blocks, s, a);
  };
  return LNORM_PICK(forward_kernel, JOIN, DROP);
}

template <bool JOIN, bool DROP>
static moe_status_t backward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  Shape S = shape_of(c);
  S.in[S.n_in++] = a.dh;
  S.in[S.n_in++] = a.x;
  if (a.dres) S.in[S.n_in++] = a.dres;
  Outs outs{};
  int kinds = 0;
  outs.p[kinds++] = a.dgamma;
  if (a.dbeta) outs.p[kinds++] = a.dbeta;
  // the CTA's groups meet in shared memory at the end
  const size_t least = S.per > 1 ? (size_t)S.per * S.H * sizeof(float) : 0;
  int blocks = 0;
  const int v = vec_of(c);
  auto go = [&](auto kern) {
    return run(kern, S, dtype_size(c.dtype), least, v * dtype_size(c.dtype) <= 8, kMaxCtas, blocks, s, a,
               kinds, outs);
  };
  const moe_status_t st = a.dres ? LNORM_PICK(backward_kernel, JOIN, DROP, true)
                                 : LNORM_PICK(backward_kernel, JOIN, DROP, false);
  if (st != MOE_OK || blocks == 1) return st;
  return launch_k(column_sum_kernel, dim3(ceil_div(kinds * c.H, 32)), dim3(1024), 0, s,
                  (const float*)a.ws, blocks, kinds, c.H, outs);
}

}  // namespace lnorm

using namespace lnorm;

size_t layer_ws_bytes(const moe_layer_t& c) {
  return (size_t)rows::max_blocks(shape_of(c)) * 2 * c.H * sizeof(float);
}

moe_status_t launch_layer_norm(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  return forward<false, false>(c, a, s);
}
moe_status_t launch_layer_norm_backward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  return backward<false, false>(c, a, s);
}
moe_status_t launch_dropout_join(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  return a.drop.below ? forward<true, true>(c, a, s) : forward<true, false>(c, a, s);
}
moe_status_t launch_dropout_join_backward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  return a.drop.below ? backward<true, true>(c, a, s) : backward<true, false>(c, a, s);
}

// ------------------------------------------------------------------- dropout alone
namespace lnorm {

constexpr int kAhead = 4;  // pieces of 8 elements a thread has in flight

template <typename T, bool DROP>
__global__ void __launch_bounds__(256) dropout_kernel(const uint8_t* x, void* out, int64_t pieces,
                                                      const __grid_constant__ Drop D) {
  pdl_wait();
  pdl_trigger();
  const int64_t first = (int64_t)blockIdx.x * (256 * kAhead) + threadIdx.x;
  Chunk<T> q[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (first + i * 256 < pieces) q[i].load(x + (first + i * 256) * Chunk<T>::kBytes);
  const Philox rng = DROP ? Philox(D) : Philox();
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int64_t at = first + i * 256;
    if (at >= pieces) break;
    F2 v[4];
    q[i].get(v);
    drop_scale<DROP>(v, &rng, D, at * 8);
    q[i].set(v);
    q[i].store(out, at * 8);
  }
}

}  // namespace lnorm

moe_status_t launch_dropout(const moe_layer_t& c, const Drop& d, const void* x, void* out,
                            cudaStream_t s) {
  const int64_t pieces = (int64_t)c.T * (c.H / 8);
  const int64_t blocks = ceil_div64(pieces, 256 * kAhead);
  if (blocks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  auto go = [&](auto kern) {
    return launch_k(kern, dim3((unsigned)blocks), dim3(256), 0, s, (const uint8_t*)x, out, pieces, d);
  };
  if (c.dtype == MOE_BF16) return d.below ? go(dropout_kernel<bf, true>) : go(dropout_kernel<bf, false>);
  return d.below ? go(dropout_kernel<float, true>) : go(dropout_kernel<float, false>);
}

}  // namespace moe
