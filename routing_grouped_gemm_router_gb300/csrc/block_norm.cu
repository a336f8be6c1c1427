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
// Every row is read once and written once, so HBM bounds all of them. A row stays in the
// registers of one group of threads between its two reductions (the reductions' results are
// needed before anything can be written); sums are fp32. Column sums over tokens (the weights'
// and a shared channel gate's gradients) are kept in registers by each group over all its rows,
// written once as partial rows, and added by a second kernel in a fixed order: no atomics, the
// same bits every run.
#include "train.cuh"

namespace moe {
namespace bnorm {

constexpr int kMaxVec = 2;  // chunks of 8 elements a thread holds

// Eight consecutive elements of a row as fp32.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    q = __ldg((const uint4*)((const __nv_bfloat16*)p + i));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const { Vec<__nv_bfloat16>::unpack(q, f); }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[8]) {
    *(uint4*)((__nv_bfloat16*)p + i) = Vec<__nv_bfloat16>::pack(f);
  }
  // the values as they are stored
  static __device__ __forceinline__ void round(float (&f)[8]) {
    Vec<__nv_bfloat16>::unpack(Vec<__nv_bfloat16>::pack(f), f);
  }
};
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = __ldg((const float4*)((const float*)p + i));
    b = __ldg((const float4*)((const float*)p + i) + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[8]) {
    float4* o = (float4*)((float*)p + i);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  static __device__ __forceinline__ void round(float (&)[8]) {}
};

__device__ __forceinline__ void load_f8(const float* p, int64_t i, float (&f)[8]) {
  Chunk<float> c;
  c.load(p, i);
  c.get(f);
}

// How a row is spread: `group` threads (a multiple of 32) a row, chunk c of the row held by
// thread c % group; a block holds blockDim / group rows.
struct Shape {
  int T, H, chunks, group, per_block;  // per_block: rows a block works on at once
  float scale, offset, eps, inv_h;
  int gate;
};

// Sums of N values over a row's group, in every thread of it. Every thread of the block calls
// it, whether its row exists or not. red: two buffers of [32 warps][N], used in turn, so that
// one barrier a reduction is enough.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int group, float* red, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_total(v[i]);
  if (group == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* buf = red + turn * 32 * 2;
  turn ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[warp * 2 + i] = v[i];
  }
  __syncthreads();
  const int w = group >> 5, first = warp / w * w;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_total(lane < w ? buf[(first + lane) * 2 + i] : 0.f);
}

// ------------------------------------------------------------------- forward
// JOIN: out = x + scale gate u, then (if gamma_next) the next norm; otherwise the norm of x.
template <typename T, int VPT, bool JOIN>
__global__ void __launch_bounds__(1024) forward_kernel(const Shape S, const BlockNormArgs A) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[2 * 32 * 2];
  int turn = 0;
  const int g = threadIdx.x % S.group;
  const int64_t t = (int64_t)blockIdx.x * S.per_block + threadIdx.x / S.group;
  const bool live = t < S.T;
  const int64_t row = (live ? t : 0) * S.H;
  const bool next = !JOIN || A.gamma_next;
  const float* gamma_n = JOIN ? A.gamma_next : A.gamma;
  Chunk<T> xq[VPT], yq[VPT], gq[VPT];
  float o[VPT][8], ssq[1] = {0.f};
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = g + v * S.group;
    if (c >= S.chunks) continue;
    if (JOIN) yq[v].load(A.y, row + c * 8);
    xq[v].load(A.x, row + c * 8);
    if (JOIN && S.gate == MOE_GATE_FULL) gq[v].load(A.gate, row + c * 8);
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (g + v * S.group >= S.chunks) continue;
    if (JOIN) yq[v].get(o[v]); else xq[v].get(o[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ssq[0] = fmaf(o[v][i], o[v][i], ssq[0]);
  }
  group_sum<1>(ssq, S.group, red, turn);
  float r = rsqrtf(ssq[0] * S.inv_h + S.eps);
  if (JOIN) {
    if (live && g == 0) A.rstd_y[t] = r;
    const float st = S.gate == MOE_GATE_TOKEN ? S.scale * __ldg((const float*)A.gate + (live ? t : 0))
                                              : S.scale;
    ssq[0] = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (c >= S.chunks) continue;
      float ga[8], x[8], gt[8];
      load_f8(A.gamma, c * 8, ga);
      xq[v].get(x);
      if (S.gate == MOE_GATE_FULL) gq[v].get(gt);
      if (S.gate == MOE_GATE_CHANNEL) load_f8((const float*)A.gate, c * 8, gt);
      const bool each = S.gate == MOE_GATE_FULL || S.gate == MOE_GATE_CHANNEL;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = o[v][i] * r * (S.offset + ga[i]);
        o[v][i] = fmaf(each ? st * gt[i] : st, u, x[i]);
      }
      if (live) Chunk<T>::store(A.out, row + c * 8, o[v]);
      Chunk<T>::round(o[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ssq[0] = fmaf(o[v][i], o[v][i], ssq[0]);
    }
    if (!next) return;
    group_sum<1>(ssq, S.group, red, turn);
    r = rsqrtf(ssq[0] * S.inv_h + S.eps);
  }
  if (!live) return;
  if (g == 0) A.rstd_out[t] = r;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = g + v * S.group;
    if (c >= S.chunks) continue;
    float ga[8];
    load_f8(gamma_n, c * 8, ga);
#pragma unroll
    for (int i = 0; i < 8; ++i) ga[i] = o[v][i] * r * (S.offset + ga[i]);
    Chunk<T>::store(A.h, row + c * 8, ga);
  }
}

// ------------------------------------------------------------------- backward
// JOIN: gradients of the join (and of the next norm, if gamma_next); otherwise of the norm of x,
// with dres added. A group takes rows t0, t0 + stride, ... and keeps the column sums.
// Partial sums go to ws[(group index) * kinds + kind][H].
template <typename T, int VPT, bool JOIN>
__global__ void __launch_bounds__(1024) backward_kernel(const Shape S, const BlockNormArgs A,
                                                        int kinds) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[2 * 32 * 2];
  int turn = 0;
  const int g = threadIdx.x % S.group;
  const int gi = blockIdx.x * S.per_block + threadIdx.x / S.group;
  const int stride = gridDim.x * S.per_block;
  const bool next = !JOIN || A.gamma_next;
  const float* gamma_n = JOIN ? A.gamma_next : A.gamma;
  const void* src = JOIN ? A.out_in : A.x;  // what the (next) norm read
  const float* rstd_n = JOIN ? A.rstd_out_in : A.rstd_y_in;
  float sn[VPT][8], sp[VPT][8], sg[VPT][8];  // sums of dh xn, of v yn, of the channel gate
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) sn[v][i] = sp[v][i] = sg[v][i] = 0.f;

  // every group of a block runs the same number of rounds: the reductions are block barriers
  const int rounds = (S.T - (int)blockIdx.x * S.per_block + stride - 1) / stride;
  for (int it = 0; it < rounds; ++it) {
    const int64_t t = gi + (int64_t)it * stride;
    const bool live = t < S.T;
    const int64_t row = (live ? t : 0) * S.H;
    Chunk<T> dq[VPT], xq[VPT], rq[VPT], yq[VPT], gq[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (c >= S.chunks) continue;
      const int64_t i = row + c * 8;
      if (next) {
        dq[v].load(A.dh, i);
        xq[v].load(src, i);
      }
      if (A.dres) rq[v].load(A.dres, i);
      if (JOIN) {
        yq[v].load(A.y, i);
        if (S.gate == MOE_GATE_FULL) gq[v].load(A.gate, i);
      }
    }
    const float rn = next ? __ldg(rstd_n + (live ? t : 0)) : 0.f;
    float d[VPT][8];
    if (next) {
      float s1[1] = {0.f};
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = g + v * S.group;
        if (c >= S.chunks) continue;
        float ga[8], x[8], dh[8];
        load_f8(gamma_n, c * 8, ga);
        xq[v].get(x);
        dq[v].get(dh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xn = x[i] * rn;
          d[v][i] = dh[i] * (S.offset + ga[i]);
          s1[0] = fmaf(d[v][i], xn, s1[0]);
          if (live) sn[v][i] = fmaf(dh[i], xn, sn[v][i]);
        }
      }
      group_sum<1>(s1, S.group, red, turn);
      const float m = s1[0] * S.inv_h;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (g + v * S.group >= S.chunks) continue;
        float x[8];
        xq[v].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[v][i] = rn * (d[v][i] - x[i] * rn * m);
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (c >= S.chunks) continue;
      if (A.dres) {
        float f[8];
        rq[v].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[v][i] = next ? d[v][i] + f[i] : f[i];
      }
      if (live) Chunk<T>::store(A.dx, row + c * 8, d[v]);
    }
    if (JOIN) {
      const float ry = __ldg(A.rstd_y_in + (live ? t : 0));
      const float tok = S.gate == MOE_GATE_TOKEN ? __ldg((const float*)A.gate + (live ? t : 0)) : 1.f;
      float s2[2] = {0.f, 0.f};  // sum of b yn; of d u (the token gate's gradient)
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = g + v * S.group;
        if (c >= S.chunks) continue;
        float y[8], ga[8], gt[8], dg[8];
        yq[v].get(y);
        load_f8(A.gamma, c * 8, ga);
        if (S.gate == MOE_GATE_FULL) gq[v].get(gt);
        if (S.gate == MOE_GATE_CHANNEL) load_f8((const float*)A.gate, c * 8, gt);
        const bool each = S.gate == MOE_GATE_FULL || S.gate == MOE_GATE_CHANNEL;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float yn = y[i] * ry, gp = S.offset + ga[i], sd = S.scale * d[v][i];
          const float vv = sd * (each ? gt[i] : tok);
          dg[i] = sd * yn * gp;
          if (live) {
            sp[v][i] = fmaf(vv, yn, sp[v][i]);
            sg[v][i] += dg[i];
          }
          s2[1] += dg[i];
          d[v][i] = vv * gp;  // b
          s2[0] = fmaf(d[v][i], yn, s2[0]);
        }
        if (live && S.gate == MOE_GATE_FULL) Chunk<T>::store(A.dgate, row + c * 8, dg);
      }
      group_sum<2>(s2, S.group, red, turn);
      const float m = s2[0] * S.inv_h;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = g + v * S.group;
        if (c >= S.chunks) continue;
        float y[8];
        yq[v].get(y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = ry * (d[v][i] - y[i] * ry * m);
        if (live) Chunk<T>::store(A.dy, row + c * 8, y);
      }
      if (live && g == 0 && S.gate == MOE_GATE_TOKEN) ((float*)A.dgate)[t] = s2[1];
    }
  }
  float* part = A.ws + (int64_t)gi * kinds * S.H;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = g + v * S.group;
    if (c >= S.chunks) continue;
    float* p = part + c * 8;
    if (JOIN) {
      Chunk<float>::store(p, 0, sp[v]);
      p += S.H;
    }
    if (next) {
      Chunk<float>::store(p, 0, sn[v]);
      p += S.H;
    }
    if (JOIN && S.gate == MOE_GATE_CHANNEL) Chunk<float>::store(p, 0, sg[v]);
  }
}

// Column sums of the partial rows: part[rows][kinds][H] -> out[kind][H]. A block takes 32
// columns; its 8 warps add every eighth row, then their sums are added in order.
struct Outs {
  float* p[3];
};
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ part, int rows,
                                                         int kinds, int H, const Outs out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sh[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t width = (int64_t)kinds * H;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < width) {
#pragma unroll 8
    for (int r = warp; r < rows; r += 8) s += part[r * width + col];
  }
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < width) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sh[i][lane];
    out.p[col / H][col % H] = s;
  }
}

// Threads a row: one chunk of 8 elements each up to 1024 chunks, two beyond (up to H 16384);
// a block is at least 128 threads, so short rows share one.
static Shape shape_of(const moe_block_t& c, int vpt) {
  Shape s{};
  s.T = c.T;
  s.H = c.H;
  s.chunks = c.H / 8;
  s.group = ceil_div(ceil_div(s.chunks, vpt), 32) * 32;
  s.per_block = std::max(1, 128 / s.group);
  s.scale = c.scale;
  s.offset = c.offset;
  s.eps = c.eps;
  s.inv_h = 1.0f / (float)c.H;
  s.gate = c.gate_kind;
  return s;
}
static int vec_of(const moe_block_t& c) { return c.H / 8 <= 1024 ? 1 : (c.H / 8 <= 2048 ? 2 : 4); }

// Groups the backward kernels run: as many as fit at once, never more than rows.
static int backward_blocks(const Shape& s) {
  const int threads = s.group * s.per_block;
  const int resident = num_sms() * std::max(1, 1024 / threads);
  return std::min(ceil_div(s.T, s.per_block), resident);
}

template <bool JOIN>
static moe_status_t forward(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  const int vpt = vec_of(c);
  const Shape S = shape_of(c, vpt);
  auto go = [&](auto kern) {
    return launch_k(kern, dim3((unsigned)ceil_div(c.T, S.per_block)), dim3(S.group * S.per_block), 0,
                    s, S, a);
  };
  if (c.dtype == MOE_BF16)
    return vpt == 1 ? go(forward_kernel<__nv_bfloat16, 1, JOIN>)
           : vpt == 2 ? go(forward_kernel<__nv_bfloat16, 2, JOIN>)
                      : go(forward_kernel<__nv_bfloat16, 4, JOIN>);
  return vpt == 1 ? go(forward_kernel<float, 1, JOIN>)
         : vpt == 2 ? go(forward_kernel<float, 2, JOIN>) : go(forward_kernel<float, 4, JOIN>);
}

template <bool JOIN>
static moe_status_t backward(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  const int vpt = vec_of(c);
  const Shape S = shape_of(c, vpt);
  const int blocks = backward_blocks(S);
  Outs outs{};
  int kinds = 0;
  if (JOIN) outs.p[kinds++] = a.dgamma;
  if (!JOIN) outs.p[kinds++] = a.dgamma;
  if (JOIN && a.gamma_next) outs.p[kinds++] = a.dgamma_next;
  if (JOIN && c.gate_kind == MOE_GATE_CHANNEL) outs.p[kinds++] = (float*)a.dgate;
  auto go = [&](auto kern) {
    return launch_k(kern, dim3(blocks), dim3(S.group * S.per_block), 0, s, S, a, kinds);
  };
  moe_status_t st;
  if (c.dtype == MOE_BF16)
    st = vpt == 1 ? go(backward_kernel<__nv_bfloat16, 1, JOIN>)
         : vpt == 2 ? go(backward_kernel<__nv_bfloat16, 2, JOIN>)
                    : go(backward_kernel<__nv_bfloat16, 4, JOIN>);
  else
    st = vpt == 1 ? go(backward_kernel<float, 1, JOIN>)
         : vpt == 2 ? go(backward_kernel<float, 2, JOIN>) : go(backward_kernel<float, 4, JOIN>);
  if (st != MOE_OK) return st;
  return launch_k(column_sum_kernel, dim3(ceil_div(kinds * c.H, 32)), dim3(256), 0, s,
                  (const float*)a.ws, blocks * S.per_block, kinds, c.H, outs);
}

}  // namespace bnorm

using namespace bnorm;

size_t block_norm_ws_bytes(const moe_block_t& c) {
  const Shape S = shape_of(c, vec_of(c));
  return (size_t)backward_blocks(S) * S.per_block * 3 * c.H * sizeof(float);
}

moe_status_t launch_block_norm(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  return forward<false>(c, a, s);
}
moe_status_t launch_block_join(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  return forward<true>(c, a, s);
}
moe_status_t launch_block_norm_backward(const moe_block_t& c, const BlockNormArgs& a,
                                        cudaStream_t s) {
  return backward<false>(c, a, s);
}
moe_status_t launch_block_join_backward(const moe_block_t& c, const BlockNormArgs& a,
                                        cudaStream_t s) {
  return backward<true>(c, a, s);
}

}  // namespace moe
