// block_norm.cu — the norms before and after a block, fused with its gate and residual scale,
// and their gradients (moe_block_norm, moe_block_join and their backward calls).
//
// With r(v) = (mean(v^2) + eps)^-1/2, gp = offset + gamma, gn = offset + gamma_next:
//   norm   h = x r(x) gn
//   join   u = y r(y) gp;  out = x + scale gate u;  h = out r(out) gn
//   back   xn = out r(out), a = dh gn:  d = dres + r(out) (a - xn mean(a xn))
//          yn = y r(y), v = scale d gate, b = v gp:  dy = r(y) (b - yn mean(b yn)),  dx = d
//          dgamma = sum_t v yn;  dgamma_next = sum_t dh xn;  dgate = scale d u, summed over
//          what shares the gate.
// Every row is read once and written once, so HBM bounds all of them. Persistent CTAs take R
// consecutive rows at a time (R > 1 where rows are short), a group of threads a row; each thread
// copies the pieces of its next rows into shared memory asynchronously (cp.async, its own pieces
// alone, so no barrier guards them) while it works on the current row from registers, so loads are
// in flight through the reductions that a row has to wait for. Sums are fp32. Column sums over
// tokens (the weights' and a shared channel gate's gradients) stay in registers over all of a
// thread's rows, are added over the CTA's groups, written as one partial row a CTA, and added by a
// second kernel in a fixed order: no atomics, the same bits every run.
#include "row_ring.cuh"

namespace moe {
namespace bnorm {

using namespace rows;

// Threads of an instance's CTA at most: 448 leave the backward kernels 144 registers.
template <int VPT>
constexpr int kThreadsOf = VPT == 2 ? 448 : kMaxThreads;

// ------------------------------------------------------------------- forward
// JOIN: out = x + scale gate u, then (if gamma_next) the next norm; otherwise the norm of x.
// Row tensors: JOIN y, x, (full gate); otherwise x.
template <typename T, int VPT, bool JOIN, int GATE>
__global__ void __launch_bounds__(kThreadsOf<VPT>, VPT <= 2 ? 2 : 1)
    forward_kernel(const __grid_constant__ Shape S,
                                                              const BlockNormArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Reducer red;
  const int local = threadIdx.x / S.group, g = threadIdx.x - local * S.group;
  Ring<T, VPT, 3> ring(S, smem, local, g);
  pdl_wait();
  pdl_trigger();
  ring.start();
  int turn = 0;
  const bool next = !JOIN || A.gamma_next;
  const float* gamma_n = JOIN ? A.gamma_next : A.gamma;
  const F2 offset = dup(S.offset);
  for (int u = blockIdx.x; u < S.units; u += gridDim.x) {
    const int t = u * S.per + local;
    const bool live = t < S.T;
    const int tl = live ? t : 0;
    const int64_t row = (int64_t)tl * S.H;
    ring.wait();
    Chunk<T> xq[VPT], gq[VPT];
    F2 o[VPT][4], sq = dup(0.f);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!ring.has[v] || !live) continue;
      Chunk<T> q;
      ring.get(q, 0, v, tl);
      if (JOIN) ring.get(xq[v], 1, v, tl);
      if (GATE == MOE_GATE_FULL) ring.get(gq[v], 2, v, tl);
      q.get(o[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = fma2(o[v][i], o[v][i], sq);
    }
    float ssq[1] = {both(sq)};
    group_sum<1>(ssq, S.group, red, turn);
    ring.refill(u);
    float r = rsqrtf(ssq[0] * S.inv_h + S.eps);
    if (JOIN) {
      if (live && g == 0) A.rstd_y[t] = r;
      const F2 sr = dup(r * (GATE == MOE_GATE_TOKEN ? S.scale * __ldg((const float*)A.gate + tl)
                                                    : S.scale));
      sq = dup(0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = g + v * S.group;
        if (!ring.has[v] || !live) continue;
        F2 ga[4], x[4], gt[4];
        load_w(A.gamma, c * 8, ga);
        xq[v].get(x);
        if (GATE == MOE_GATE_FULL) gq[v].get(gt);
        if (GATE == MOE_GATE_CHANNEL) load_w((const float*)A.gate, c * 8, gt);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          F2 u = o[v][i] * (offset + ga[i]);
          if (GATE == MOE_GATE_FULL || GATE == MOE_GATE_CHANNEL) u = u * gt[i];
          o[v][i] = fma2(u, sr, x[i]);
        }
        Chunk<T> q;
        q.set(o[v]);
        q.store(A.out, row + c * 8);
        q.get(o[v]);  // the next norm reads what is stored
#pragma unroll
        for (int i = 0; i < 4; ++i) sq = fma2(o[v][i], o[v][i], sq);
      }
      if (!next) continue;
      ssq[0] = both(sq);
      group_sum<1>(ssq, S.group, red, turn);
      r = rsqrtf(ssq[0] * S.inv_h + S.eps);
    }
    if (!live) continue;
    if (g == 0) A.rstd_out[t] = r;
    const F2 rr = dup(r);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!ring.has[v]) continue;
      F2 ga[4];
      load_w(gamma_n, c * 8, ga);
#pragma unroll
      for (int i = 0; i < 4; ++i) ga[i] = o[v][i] * rr * (offset + ga[i]);
      Chunk<T> q;
      q.set(ga);
      q.store(A.h, row + c * 8);
    }
  }
}

// ------------------------------------------------------------------- backward
// JOIN: gradients of the join (and of the next norm, if gamma_next); otherwise of the norm of x,
// with dres added. BOTH: a next norm and dres are both there, as everywhere inside a stack (known at
// compile time that takes 7 to 24 % off: 8192 x 4096 with a token gate 88 -> 82 us, 8192 x 7168 with a
// channel gate 215 -> 164). Row tensors, those that are there: dh, what the norm read (x or out), dres,
// y, full gate. A token gate (and the scale) is a factor of a whole row and a channel gate's scale
// one of a whole column, so they are taken out of the sums:
//   q = sum d yn gp (gate):  dgate_token = scale q,  mean(b yn) = scale (gate) q / H;
// and with d = d0 - m x, m from the next norm's own reduction, q = sum d0 yn gp - m sum x yn gp: the
// three sums of a row are taken together, and one barrier a row is enough.
template <typename T, int VPT, bool JOIN, int GATE, bool BOTH>
__global__ void __launch_bounds__(kThreadsOf<VPT>)
    backward_kernel(const __grid_constant__ Shape S,
                                                               const BlockNormArgs A, int kinds,
                                                               const Outs outs) {
  constexpr bool EACH = GATE == MOE_GATE_FULL || GATE == MOE_GATE_CHANNEL;
  constexpr bool CHANNEL = GATE == MOE_GATE_CHANNEL;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Reducer red;
  const int local = threadIdx.x / S.group, g = threadIdx.x - local * S.group;
  Ring<T, VPT, kMaxIn> ring(S, smem, local, g);
  pdl_wait();
  pdl_trigger();
  ring.start();
  int turn = 0;
  const bool next = BOTH || !JOIN || A.gamma_next, res = BOTH || A.dres;
  const float* gamma_n = JOIN ? A.gamma_next : A.gamma;
  const float* rstd_n = JOIN ? A.rstd_out_in : A.rstd_y_in;
  const int i_res = next ? 2 : 0, i_y = i_res + (res ? 1 : 0);
  const F2 offset = dup(S.offset), zero = dup(0.f);
  F2 sn[VPT][4], sp[JOIN ? VPT : 1][4], sg[CHANNEL ? VPT : 1][4];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sn[v][i] = zero;
      if (JOIN) sp[v][i] = zero;
      if (CHANNEL) sg[v][i] = zero;
    }

  // a row's scalars are asked for one row ahead: nothing else hides their way from L2
  float rn_next = 0.f, ry_next = 0.f, tok_next = 1.f;
  auto scalars = [&](int t) {
    if (t >= S.T) t = 0;
    if (next) rn_next = __ldg(rstd_n + t);
    if (JOIN) ry_next = __ldg(A.rstd_y_in + t);
    if (GATE == MOE_GATE_TOKEN) tok_next = __ldg((const float*)A.gate + t);
  };
  scalars(blockIdx.x * S.per + local);
  for (int u = blockIdx.x; u < S.units; u += gridDim.x) {
    const int t = u * S.per + local;
    const bool live = t < S.T;
    const int tl = live ? t : 0;
    const int64_t row = (int64_t)tl * S.H;
    const float rn = rn_next, ry = ry_next, tok = S.scale * tok_next;
    scalars(t + gridDim.x * S.per);
    ring.wait();
    const F2 rn2 = dup(rn), ry2 = dup(ry);
    Chunk<T> xq[VPT], yq[VPT], gq[VPT];
    F2 d[VPT][4], s1 = zero, q0 = zero, q1 = zero;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!ring.has[v] || !live) continue;
      F2 x[4];
      if (next) {
        Chunk<T> dq;
        ring.get(dq, 0, v, tl);
        ring.get(xq[v], 1, v, tl);
        F2 ga[4];
        load_w(gamma_n, c * 8, ga);
        xq[v].get(x);
        dq.get(d[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 xn = x[i] * rn2;
          sn[v][i] = fma2(d[v][i], xn, sn[v][i]);
          d[v][i] = d[v][i] * (offset + ga[i]);
          s1 = fma2(d[v][i], xn, s1);
          d[v][i] = d[v][i] * rn2;
        }
      }
      if (res) {
        Chunk<T> rq;
        F2 f[4];
        ring.get(rq, i_res, v, tl);
        rq.get(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] = next ? d[v][i] + f[i] : f[i];
      }
      if (JOIN) {
        F2 y[4], ga[4], gt[4];
        ring.get(yq[v], i_y, v, tl);
        if (GATE == MOE_GATE_FULL) {
          ring.get(gq[v], i_y + 1, v, tl);
          gq[v].get(gt);
        }
        if (CHANNEL) load_w((const float*)A.gate, c * 8, gt);
        yq[v].get(y);
        load_w(A.gamma, c * 8, ga);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          F2 w = y[i] * (offset + ga[i]);
          if (EACH) w = w * gt[i];
          q0 = fma2(d[v][i], w, q0);
          if (next) q1 = fma2(x[i], w, q1);
        }
      }
    }
    float s[3] = {both(s1), both(q0), both(q1)};
    if (JOIN) group_sum<3>(s, S.group, red, turn);
    else group_sum<1>(s, S.group, red, turn);
    ring.refill(u);
    const float m = -s[0] * S.inv_h * rn * rn;   // dx = d + m x
    const float q = (s[1] + m * s[2]) * ry;      // sum of dx yn gp (gate)
    const F2 m2 = dup(m), my = dup(-tok * q * S.inv_h * ry * ry), f = dup(tok * ry);
    if (JOIN && GATE == MOE_GATE_TOKEN && live && g == 0) ((float*)A.dgate)[t] = S.scale * q;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!ring.has[v] || !live) continue;
      if (next) {
        F2 x[4];
        xq[v].get(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[v][i] = fma2(x[i], m2, d[v][i]);
      }
      Chunk<T> o;
      o.set(d[v]);
      o.store(A.dx, row + c * 8);
      if (JOIN) {
        F2 y[4], ga[4], gt[4], dg[4];
        yq[v].get(y);
        load_w(A.gamma, c * 8, ga);
        if (GATE == MOE_GATE_FULL) gq[v].get(gt);
        if (CHANNEL) load_w((const float*)A.gate, c * 8, gt);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 gp = offset + ga[i], e = d[v][i] * y[i] * ry2;
          if (EACH) {
            sp[v][i] = fma2(e, gt[i], sp[v][i]);  // times scale at the end
            dg[i] = e * gp;
            if (CHANNEL) sg[v][i] = sg[v][i] + dg[i];
            if (GATE == MOE_GATE_FULL) dg[i] = dg[i] * dup(S.scale);
            d[v][i] = d[v][i] * gt[i];
          } else {
            sp[v][i] = fma2(e, dup(tok), sp[v][i]);
          }
          y[i] = fma2(y[i], my, d[v][i] * gp * f);
        }
        if (GATE == MOE_GATE_FULL) {
          o.set(dg);
          o.store(A.dgate, row + c * 8);
        }
        o.set(y);
        o.store(A.dy, row + c * 8);
      }
    }
  }

  int kind = 0;
  auto leave = [&](const F2 (&s)[VPT][4], float factor) {
    leave_columns<VPT>(S, smem, local, g, s, kind++, kinds, factor, A.ws, outs);
  };
  if constexpr (JOIN) leave(sp, EACH ? S.scale : 1.f);
  if (next) leave(sn, 1.f);
  if constexpr (CHANNEL) leave(sg, S.scale);
}

// Chunks of 8 elements a thread holds. More of them share the fixed cost of a warp's row (the
// reductions), until registers run out: the join's kernels hold four rows and their sums. Measured at
// 8192 rows of bf16, two against four chunks, us: join of 4096 channels 51 and 60, its gradient 84 and
// 119; of 7168 channels 90 and 98, 146 and 193. Norm of 5120 channels 35.3 and 34.7, its gradient 67 and 70;
// of 7168 50 and 54, 103 and 93: one rule for both directions, for the gradient's sake.
static int vec_of(const moe_block_t& c, bool join) {
  const int chunks = c.H / 8;
  const int two = join || c.dtype == MOE_F32 ? 896 : 512;
  return chunks <= 32 ? 1 : chunks <= two ? 2 : chunks <= 2048 ? 4 : 8;
}
static Shape shape_of(const moe_block_t& c, bool join) {
  Shape s{};
  s.T = c.T;
  s.H = c.H;
  s.chunks = c.H / 8;
  s.group = ceil_div(ceil_div(s.chunks, vec_of(c, join)), 32) * 32;
  s.per = std::min(c.T, std::max(1, 256 / s.group));
  s.units = ceil_div(c.T, s.per);
  s.scale = c.scale;
  s.offset = c.offset;
  s.eps = c.eps;
  s.inv_h = 1.0f / (float)c.H;
  return s;
}

using bf = __nv_bfloat16;

// The kernel instance of a dtype and a row length.
#define BNORM_PICK(name, ...)                                                       \
  (c.dtype == MOE_BF16 ? (v == 1   ? go(name<bf, 1, __VA_ARGS__>)                   \
                          : v == 2 ? go(name<bf, 2, __VA_ARGS__>)                   \
                          : v == 4 ? go(name<bf, 4, __VA_ARGS__>)                   \
                                   : go(name<bf, 8, __VA_ARGS__>))                  \
                       : (v == 1   ? go(name<float, 1, __VA_ARGS__>)                \
                          : v == 2 ? go(name<float, 2, __VA_ARGS__>)                \
                          : v == 4 ? go(name<float, 4, __VA_ARGS__>)                \
                                   : go(name<float, 8, __VA_ARGS__>)))

template <bool JOIN, int GATE>
static moe_status_t forward(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  Shape S = shape_of(c, JOIN);
  if (JOIN) S.in[S.n_in++] = a.y;
  S.in[S.n_in++] = a.x;
  if (GATE == MOE_GATE_FULL) S.in[S.n_in++] = a.gate;
  int blocks = 0;
  const int v = vec_of(c, JOIN);
  auto go = [&](auto kern) { return run(kern, S, dtype_size(c.dtype), 0, v * dtype_size(c.dtype) <= 8, 8, blocks, s, a); };
  return BNORM_PICK(forward_kernel, JOIN, GATE);
}

template <bool JOIN, int GATE>
static moe_status_t backward(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  Shape S = shape_of(c, JOIN);
  const bool next = !JOIN || a.gamma_next;
  if (next) {
    S.in[S.n_in++] = a.dh;
    S.in[S.n_in++] = JOIN ? a.out_in : a.x;
  }
  if (a.dres) S.in[S.n_in++] = a.dres;
  if (JOIN) S.in[S.n_in++] = a.y;
  if (GATE == MOE_GATE_FULL) S.in[S.n_in++] = a.gate;
  Outs outs{};
  int kinds = 0;
  outs.p[kinds++] = a.dgamma;
  if (JOIN && next) outs.p[kinds++] = a.dgamma_next;
  if (GATE == MOE_GATE_CHANNEL) outs.p[kinds++] = (float*)a.dgate;
  // the CTA's groups meet in shared memory at the end
  const size_t least = S.per > 1 ? (size_t)S.per * S.H * sizeof(float) : 0;
  int blocks = 0;
  const int v = vec_of(c, JOIN);
  auto go = [&](auto kern) {
    return run(kern, S, dtype_size(c.dtype), least, v * dtype_size(c.dtype) <= 8, kMaxCtas, blocks, s, a,
               kinds, outs);
  };
  moe_status_t st;
  if constexpr (JOIN) {
    st = next && a.dres ? BNORM_PICK(backward_kernel, true, GATE, true)
                        : BNORM_PICK(backward_kernel, true, GATE, false);
  } else {
    st = BNORM_PICK(backward_kernel, false, MOE_GATE_NONE, false);
  }
  if (st != MOE_OK || blocks == 1) return st;
  return launch_column_sum(a.ws, blocks, kinds, c.H, outs, s);
}

}  // namespace bnorm

using namespace bnorm;

size_t block_norm_ws_bytes(const moe_block_t& c) {
  // the same size for both kinds of call
  const int rows = std::max(max_blocks(shape_of(c, false)), max_blocks(shape_of(c, true)));
  return (size_t)rows * 3 * c.H * sizeof(float);
}

moe_status_t launch_block_norm(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  return forward<false, MOE_GATE_NONE>(c, a, s);
}
moe_status_t launch_block_join(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  switch (c.gate_kind) {
    case MOE_GATE_NONE: return forward<true, MOE_GATE_NONE>(c, a, s);
    case MOE_GATE_CHANNEL: return forward<true, MOE_GATE_CHANNEL>(c, a, s);
    case MOE_GATE_TOKEN: return forward<true, MOE_GATE_TOKEN>(c, a, s);
    default: return forward<true, MOE_GATE_FULL>(c, a, s);
  }
}
moe_status_t launch_block_norm_backward(const moe_block_t& c, const BlockNormArgs& a,
                                        cudaStream_t s) {
  return backward<false, MOE_GATE_NONE>(c, a, s);
}
moe_status_t launch_block_join_backward(const moe_block_t& c, const BlockNormArgs& a,
                                        cudaStream_t s) {
  switch (c.gate_kind) {
    case MOE_GATE_NONE: return backward<true, MOE_GATE_NONE>(c, a, s);
    case MOE_GATE_CHANNEL: return backward<true, MOE_GATE_CHANNEL>(c, a, s);
    case MOE_GATE_TOKEN: return backward<true, MOE_GATE_TOKEN>(c, a, s);
    default: return backward<true, MOE_GATE_FULL>(c, a, s);
  }
}

}  // namespace moe
