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
#include "tc_ptx.cuh"
#include "train.cuh"

namespace moe {
namespace bnorm {

using namespace ptx;

constexpr int kMaxIn = 5;         // row tensors a kernel reads
constexpr int kMaxStages = 3;
constexpr int kMaxThreads = 512;  // of a CTA
// Threads of an instance's CTA at most: 448 leave the backward kernels 144 registers.
template <int VPT>
constexpr int kThreadsOf = VPT == 2 ? 448 : kMaxThreads;
constexpr int kRingBudget = 128 * 1024;  // bytes of rows in flight an SM; the rest is L1 (the weights)

// Packed pairs (F2): the arithmetic of a row, not only its bytes, has to fit in the time HBM leaves
// (an element passes through about 20 operations forward and 30 backward), and packed operations
// halve it.
__device__ __forceinline__ F2 dup(float s) { return f2(s, s); }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float both(F2 a) {
  float lo, hi;
  split(a, lo, hi);
  return lo + hi;
}

// Eight consecutive elements of a row, as they are stored and as four pairs; from shared or
// global memory.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 q;
  static constexpr int kBytes = 16;
  __device__ __forceinline__ void load(const uint8_t* p) { q = __ldcs((const uint4*)p); }
  __device__ __forceinline__ void load_shared(const uint8_t* p) { q = *(const uint4*)p; }
  __device__ __forceinline__ void get(F2 (&f)[4]) const {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void set(const F2 (&f)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      split(f[i], lo, hi);
      u[i] = pack_bf16(lo, hi);
    }
    q = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    *(uint4*)((__nv_bfloat16*)p + i) = q;
  }
};
template <>
struct Chunk<float> {
  F2 v[4];
  static constexpr int kBytes = 32;
  __device__ __forceinline__ void set(const float4& a, const float4& b) {
    v[0] = f2(a.x, a.y); v[1] = f2(a.z, a.w); v[2] = f2(b.x, b.y); v[3] = f2(b.z, b.w);
  }
  __device__ __forceinline__ void load(const uint8_t* p) {
    set(__ldcs((const float4*)p), __ldcs((const float4*)p + 1));
  }
  __device__ __forceinline__ void load_shared(const uint8_t* p) {
    set(*(const float4*)p, *((const float4*)p + 1));
  }
  __device__ __forceinline__ void get(F2 (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i];
  }
  __device__ __forceinline__ void set(const F2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f[i];
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) split(v[k], f[2 * k], f[2 * k + 1]);
    float4* o = (float4*)((float*)p + i);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Eight fp32 weights (or shared gates), from L1 after the CTA's first row.
__device__ __forceinline__ void load_w(const float* p, int i, F2 (&f)[4]) {
  const float4 a = __ldg((const float4*)(p + i)), b = __ldg((const float4*)(p + i) + 1);
  f[0] = f2(a.x, a.y); f[1] = f2(a.z, a.w); f[2] = f2(b.x, b.y); f[3] = f2(b.z, b.w);
}

// How rows are spread: `group` threads (a multiple of 32) a row, chunk c of the row held by
// thread c % group; a CTA works on `per` consecutive rows at once (a unit).
struct Shape {
  int T, H, chunks, group, per, units;
  float scale, offset, eps, inv_h;
  int n_in;           // row tensors read
  int stages;
  const void* in[kMaxIn];
};

// Sums of N values over a row's group, in every thread of it. Every thread of the CTA calls it,
// whether its row exists or not. Two buffers used in turn make one barrier a reduction enough.
struct Reducer {
  float buf[2][3][kMaxThreads / 32];
};
template <int N, int M>
__device__ __forceinline__ void group_sum(float (&v)[M], int group, Reducer& red, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_total(v[i]);
  if (group == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto& buf = red.buf[turn];
  turn ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i][warp] = v[i];
  }
  __syncthreads();
  const int w = group >> 5, first = warp / w * w;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_total(lane < w ? buf[i][first + lane] : 0.f);
}

// A thread's pieces of its next rows. A stage holds, tensor by tensor, the CTA's rows; a thread
// writes and reads only its own chunks, so the order of its own copies is all that counts. Rows
// too long for the ring (kRinged) are read from global memory as they are used.
template <typename T, int VPT>
constexpr bool kRinged = VPT * (int)sizeof(T) <= 8;

template <typename T, int VPT, int MAXIN>
struct Ring {
  static constexpr bool on = kRinged<T, VPT>;
  const Shape& S;
  const uint8_t* mine;    // this thread's first chunk in the current stage
  uint32_t first;         // and in stage 0, as a shared address
  uint32_t tensor_bytes, stage_bytes, step;  // step: from a thread's chunk to its next
  uint32_t row_bytes, off;                   // off: its first chunk inside a row
  bool has[VPT];
  int local, stage = 0;
  __device__ __forceinline__ Ring(const Shape& S_, uint8_t* smem, int local_, int g)
      : S(S_), local(local_) {
    row_bytes = (uint32_t)S.H * sizeof(T);
    tensor_bytes = row_bytes * S.per;
    stage_bytes = tensor_bytes * S.n_in;
    step = S.group * Chunk<T>::kBytes;
    off = g * Chunk<T>::kBytes;
    mine = smem + local * row_bytes + off;
    first = su32(mine);
#pragma unroll
    for (int v = 0; v < VPT; ++v) has[v] = g + v * S.group < S.chunks;
  }
  __device__ __forceinline__ void issue(int u, int s) {  // one group of copies: unit u into stage s
    if (!on) return;
    const int t = u * S.per + local;
    if (u < S.units && t < S.T) {
      const int64_t from = (int64_t)t * row_bytes + off;
      uint32_t dst = first + s * stage_bytes;
#pragma unroll
      for (int i = 0; i < MAXIN; ++i) {
        if (i >= S.n_in) break;
        const uint8_t* src = (const uint8_t*)S.in[i] + from;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          if (has[v]) {
#pragma unroll
            for (int b = 0; b < Chunk<T>::kBytes; b += 16)
              cp_async16(dst + v * step + b, src + v * step + b, 16);
          }
        }
        dst += tensor_bytes;
      }
    }
    cp_async_commit();
  }
  __device__ __forceinline__ void start() {  // the first units of this CTA
    for (int s = 0; s < S.stages; ++s) issue(blockIdx.x + s * gridDim.x, s);
  }
  __device__ __forceinline__ void wait() {  // the oldest group has landed
    if (!on) return;
    if (S.stages == 1) cp_async_wait<0>();
    else if (S.stages == 2) cp_async_wait<1>();
    else cp_async_wait<2>();
  }
  // chunk v of tensor i in the current unit; t: its row
  __device__ __forceinline__ void get(Chunk<T>& q, int i, int v, int t) const {
    if (on) q.load_shared(mine + i * tensor_bytes + v * step);
    else q.load((const uint8_t*)S.in[i] + (int64_t)t * row_bytes + off + v * step);
  }
  // the current stage's values have been used: its next unit
  __device__ __forceinline__ void refill(int u) {
    if (!on) return;
    issue(u + S.stages * gridDim.x, stage);
    mine += stage_bytes;
    if (++stage == S.stages) {
      stage = 0;
      mine -= S.stages * stage_bytes;
    }
  }
};

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

// Where the column sums of `kinds` kinds go: the results themselves when there is one CTA.
struct Outs {
  float* p[3];
};

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

  // The CTA's column sums: its groups' sums are added in order through shared memory (the ring,
  // whose copies have all landed), then leave as a partial row, or as the result of a lone CTA.
  auto leave = [&](F2 (&s)[VPT][4], int kind, float factor) {
    float* to = gridDim.x == 1 ? outs.p[kind]
                               : A.ws + ((int64_t)blockIdx.x * kinds + kind) * S.H;
    float* all = S.per > 1 ? (float*)smem + (int64_t)local * S.H : to;
    if (S.per > 1) __syncthreads();
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (c >= S.chunks) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(s[v][i], lo, hi);
        all[c * 8 + 2 * i] = lo * factor;
        all[c * 8 + 2 * i + 1] = hi * factor;
      }
    }
    if (S.per == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < S.H; c += blockDim.x) {
      float sum = 0.f;
      for (int l = 0; l < S.per; ++l) sum += ((const float*)smem)[l * S.H + c];
      to[c] = sum;
    }
  };
  int kind = 0;
  if constexpr (JOIN) leave(sp, kind++, EACH ? S.scale : 1.f);
  if (next) leave(sn, kind++, 1.f);
  if constexpr (CHANNEL) leave(sg, kind++, S.scale);
}

// Column sums of the partial rows: part[rows][kinds][H] -> out[kind][H]. A block takes 32
// columns; each of its 32 warps adds every 32nd row, then their sums are added in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ part, int rows,
                                                          int kinds, int H, const Outs out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t width = (int64_t)kinds * H;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < width) {
#pragma unroll 8
    for (int r = warp; r < rows; r += 32) s += part[r * width + col];
  }
  sh[warp][lane] = s;
  __syncthreads();
  // warp w sums column w of the block over the 32 warps
  s = warp_total(sh[lane][warp]);
  const int64_t c = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && c < width) out.p[c / H][c % H] = s;
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

// Partial rows at most: the backward kernels' CTAs.
constexpr int kMaxCtas = 4;  // an SM
static int max_blocks(const Shape& s) { return std::min(s.units, num_sms() * kMaxCtas); }

// Fills in the ring's stages, as many as the budget of an SM's resident CTAs allows. Returns the
// CTA's dynamic shared memory.
static size_t plan_ring(Shape& s, size_t es, int ctas, bool ringed) {
  const size_t stage = (size_t)s.per * s.H * es * s.n_in;
  s.stages = 1;
  if (!ringed) return 0;
  s.stages = (int)std::min<size_t>(kMaxStages, std::max<size_t>(1, kRingBudget / ctas / stage));
  return stage * s.stages;
}

template <typename... KArgs, typename... Args>
static moe_status_t run(void (*kern)(KArgs...), Shape& S, size_t es, size_t least, bool ringed,
                        int max_ctas, int& blocks, cudaStream_t s, Args&&... args) {
  const int threads = S.group * S.per;
  // CTAs an SM: what their registers allow (asked once a kernel, size and device), shared memory
  // being divided among them
  struct Key {
    void* k;
    int dev, threads, ctas;
  };
  static thread_local Key last[8];
  static thread_local int at = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  Key* hit = nullptr;
  for (Key& k : last)
    if (k.k == (void*)kern && k.dev == dev && k.threads == threads) hit = &k;
  if (!hit) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 1024) != cudaSuccess ||
        n < 1)
      return MOE_ERR_CUDA;
    hit = &last[at++ & 7];
    *hit = {(void*)kern, dev, threads, n};
  }
  int ctas = std::min(hit->ctas, max_ctas);
  size_t smem = std::max(plan_ring(S, es, ctas, ringed), least);
  ctas = std::max(1, std::min<int>(ctas, (int)(220 * 1024 / (smem + 1024))));
  blocks = std::min(S.units, num_sms() * ctas);
  return launch_k(kern, dim3(blocks), dim3(threads), smem, s, (const Shape&)S,
                  std::forward<Args>(args)...);
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
  return launch_k(column_sum_kernel, dim3(ceil_div(kinds * c.H, 32)), dim3(1024), 0, s,
                  (const float*)a.ws, blocks, kinds, c.H, outs);
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
