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
// consecutive rows at a time (R > 1 where rows are short): one bulk copy a tensor brings them
// into shared memory, a group of threads a row takes its row into registers, and the copies of
// the CTA's next rows are issued at once, so loads are in flight through the two reductions that
// a row has to wait for. Sums are fp32. Column sums over tokens (the weights' and a shared channel
// gate's gradients) stay in registers over all of a thread's rows, are added over the CTA's groups,
// written as one partial row a CTA, and added by a second kernel in a fixed order: no atomics, the
// same bits every run.
#include "tc_ptx.cuh"
#include "train.cuh"

namespace moe {
namespace bnorm {

using namespace ptx;

__device__ int g_status;

constexpr int kMaxIn = 5;         // row tensors a kernel reads
constexpr int kMaxStages = 3;
constexpr int kMaxThreads = 512;  // of a CTA
constexpr int kRingBudget = 128 * 1024;  // bytes of rows in flight an SM; the rest is L1 (the weights)
constexpr int kMaxRing = 200 * 1024;     // of one CTA

// Eight consecutive elements of a row as fp32, from shared or global memory.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const void* row, int i) {
    q = *((const uint4*)((const __nv_bfloat16*)row + i));
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
  __device__ __forceinline__ void load(const void* row, int i) {
    a = *((const float4*)((const float*)row + i));
    b = *((const float4*)((const float*)row + i) + 1);
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

__device__ __forceinline__ void load_f8(const float* p, int i, float (&f)[8]) {
  const float4 a = __ldg((const float4*)(p + i)), b = __ldg((const float4*)(p + i) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// How rows are spread: `group` threads (a multiple of 32) a row, chunk c of the row held by
// thread c % group; a CTA works on `per` consecutive rows at once (a unit).
struct Shape {
  int T, H, chunks, group, per, units;
  float scale, offset, eps, inv_h;
  int gate;
  int n_in, ringed;   // row tensors read; the first `ringed` of them go through the ring
  int stages;
  const void* in[kMaxIn];
};

// Sums of N values over a row's group, in every thread of it. Every thread of the block calls
// it, whether its row exists or not. red: two buffers of [16 warps][2], used in turn, so that
// one barrier a reduction is enough.
struct Reducer {
  float buf[2][kMaxThreads / 32][2];
};
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int group, Reducer& red, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_total(v[i]);
  if (group == 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto& buf = red.buf[turn];
  turn ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[warp][i] = v[i];
  }
  __syncthreads();
  const int w = group >> 5, first = warp / w * w;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_total(lane < w ? buf[first + lane][i] : 0.f);
}

// The ring of units: stage s holds the rows of the ringed tensors one after another.
template <typename T>
struct Ring {
  const Shape& S;
  uint8_t* smem;
  uint64_t* full;
  volatile int* abort_flag;
  __device__ __forceinline__ size_t tensor_bytes() const {
    return (size_t)S.per * S.H * sizeof(T);
  }
  __device__ __forceinline__ void init() {
    if (threadIdx.x == 0) {
      for (int s = 0; s < S.stages; ++s) mbar_init(&full[s], 1);
      *abort_flag = 0;
      mbar_init_fence();
    }
    __syncthreads();
  }
  __device__ __forceinline__ void issue(int it) {  // one thread: the CTA's it-th unit
    const int64_t u = blockIdx.x + (int64_t)it * gridDim.x;
    if (u >= S.units || S.ringed == 0) return;
    const int s = it % S.stages;
    const int rows = (int)min((int64_t)S.per, S.T - u * S.per);
    const uint32_t bytes = (uint32_t)((size_t)rows * S.H * sizeof(T));
    mbar_expect_tx(&full[s], bytes * S.ringed);
    uint8_t* dst = smem + s * S.ringed * tensor_bytes();
    for (int i = 0; i < S.ringed; ++i) {
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
              su32(dst + i * tensor_bytes())),
          "l"((const T*)S.in[i] + u * S.per * S.H), "r"(bytes), "r"(su32(&full[s]))
          : "memory");
    }
  }
  __device__ __forceinline__ bool wait(int it) {
    if (S.ringed == 0) return true;
    return wait_bounded(&full[it % S.stages], (uint32_t)(it / S.stages) & 1u, abort_flag, &g_status);
  }
  // Overdue: copies in flight get 200 us to land before the CTA's shared memory is released.
  __device__ __forceinline__ void abandon() const {
    const uint64_t t0 = gtimer();
    while (gtimer() - t0 < 200000ull) {
    }
  }
  // tensor i's row `local` of the CTA's it-th unit (row t of the tensor)
  __device__ __forceinline__ const void* row(int i, int it, int local, int64_t t) const {
    if (i < S.ringed)
      return smem + ((it % S.stages) * S.ringed + i) * tensor_bytes() +
             (size_t)local * S.H * sizeof(T);
    return (const T*)S.in[i] + t * S.H;
  }
};

struct Shared {
  uint64_t full[kMaxStages];
  int abort_flag;
  Reducer red;
};

// ------------------------------------------------------------------- forward
// JOIN: out = x + scale gate u, then (if gamma_next) the next norm; otherwise the norm of x.
// Row tensors: JOIN y, x, (full gate); otherwise x.
template <typename T, int VPT, bool JOIN>
__global__ void __launch_bounds__(kMaxThreads) forward_kernel(const __grid_constant__ Shape S,
                                                              const BlockNormArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared sh;
  Ring<T> ring{S, smem, sh.full, &sh.abort_flag};
  ring.init();
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0)
    for (int it = 0; it < S.stages; ++it) ring.issue(it);
  int turn = 0;
  const int local = threadIdx.x / S.group, g = threadIdx.x - local * S.group;
  const bool next = !JOIN || A.gamma_next;
  const bool full = JOIN && S.gate == MOE_GATE_FULL;
  const float* gamma_n = JOIN ? A.gamma_next : A.gamma;
  for (int it = 0; blockIdx.x + (int64_t)it * gridDim.x < S.units; ++it) {
    const int64_t t = (blockIdx.x + (int64_t)it * gridDim.x) * S.per + local;
    const bool live = t < S.T;
    const int64_t row = (live ? t : 0) * S.H;
    const bool arrived = ring.wait(it);
    const void* r0 = ring.row(0, it, local, live ? t : 0);
    const void* r1 = JOIN ? ring.row(1, it, local, live ? t : 0) : nullptr;
    const void* r2 = full ? ring.row(2, it, local, live ? t : 0) : nullptr;
    Chunk<T> xq[VPT], gq[VPT];
    float o[VPT][8], ssq[1] = {0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (c >= S.chunks || !live) continue;
      Chunk<T> q;
      q.load(r0, c * 8);
      if (JOIN) xq[v].load(r1, c * 8);
      if (full) gq[v].load(r2, c * 8);
      q.get(o[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ssq[0] = fmaf(o[v][i], o[v][i], ssq[0]);
    }
    if (!__syncthreads_and(arrived)) {  // the stage has been read, or a copy is overdue
      ring.abandon();
      return;
    }
    if (threadIdx.x == 0) ring.issue(it + S.stages);
    group_sum<1>(ssq, S.group, sh.red, turn);
    float r = rsqrtf(ssq[0] * S.inv_h + S.eps);
    if (JOIN) {
      if (live && g == 0) A.rstd_y[t] = r;
      const float st = S.gate == MOE_GATE_TOKEN
                           ? S.scale * __ldg((const float*)A.gate + (live ? t : 0))
                           : S.scale;
      ssq[0] = 0.f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = g + v * S.group;
        if (c >= S.chunks || !live) continue;
        float ga[8], x[8], gt[8];
        load_f8(A.gamma, c * 8, ga);
        xq[v].get(x);
        if (full) gq[v].get(gt);
        if (S.gate == MOE_GATE_CHANNEL) load_f8((const float*)A.gate, c * 8, gt);
        const bool each = full || S.gate == MOE_GATE_CHANNEL;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = o[v][i] * r * (S.offset + ga[i]);
          o[v][i] = fmaf(each ? st * gt[i] : st, u, x[i]);
        }
        Chunk<T>::store(A.out, row + c * 8, o[v]);
        Chunk<T>::round(o[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ssq[0] = fmaf(o[v][i], o[v][i], ssq[0]);
      }
      if (!next) continue;
      group_sum<1>(ssq, S.group, sh.red, turn);
      r = rsqrtf(ssq[0] * S.inv_h + S.eps);
    }
    if (!live) continue;
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
}

// Where the column sums of `kinds` kinds go: the results themselves when there is one CTA.
struct Outs {
  float* p[3];
};

// ------------------------------------------------------------------- backward
// JOIN: gradients of the join (and of the next norm, if gamma_next); otherwise of the norm of x,
// with dres added. CHANNEL: a gate shared by all tokens, whose gradient is a column sum too.
// Row tensors, those that are there: dh, what the norm read (x or out), dres, y, full gate.
template <typename T, int VPT, bool JOIN, bool CHANNEL>
__global__ void __launch_bounds__(kMaxThreads) backward_kernel(const __grid_constant__ Shape S,
                                                               const BlockNormArgs A, int kinds,
                                                               const Outs outs) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared sh;
  Ring<T> ring{S, smem, sh.full, &sh.abort_flag};
  ring.init();
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0)
    for (int it = 0; it < S.stages; ++it) ring.issue(it);
  int turn = 0;
  const int local = threadIdx.x / S.group, g = threadIdx.x - local * S.group;
  const bool next = !JOIN || A.gamma_next;
  const bool full = JOIN && S.gate == MOE_GATE_FULL;
  const float* gamma_n = JOIN ? A.gamma_next : A.gamma;
  const float* rstd_n = JOIN ? A.rstd_out_in : A.rstd_y_in;
  const int i_res = next ? 2 : 0, i_y = i_res + (A.dres ? 1 : 0);
  float sn[VPT][8], sp[JOIN ? VPT : 1][8], sg[CHANNEL ? VPT : 1][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sn[v][i] = 0.f;
      if (JOIN) sp[v][i] = 0.f;
      if (CHANNEL) sg[v][i] = 0.f;
    }

  for (int it = 0; blockIdx.x + (int64_t)it * gridDim.x < S.units; ++it) {
    const int64_t t = (blockIdx.x + (int64_t)it * gridDim.x) * S.per + local;
    const bool live = t < S.T;
    const int64_t tl = live ? t : 0, row = tl * S.H;
    const bool arrived = ring.wait(it);
    const void *rd = nullptr, *rx = nullptr, *rr = nullptr, *ry_ = nullptr, *rg = nullptr;
    if (next) {
      rd = ring.row(0, it, local, tl);
      rx = ring.row(1, it, local, tl);
    }
    if (A.dres) rr = ring.row(i_res, it, local, tl);
    if (JOIN) ry_ = ring.row(i_y, it, local, tl);
    if (full) rg = ring.row(i_y + 1, it, local, tl);
    const float rn = next ? __ldg(rstd_n + tl) : 0.f;
    const float ry = JOIN ? __ldg(A.rstd_y_in + tl) : 0.f;
    const float tok = JOIN && S.gate == MOE_GATE_TOKEN ? __ldg((const float*)A.gate + tl) : 1.f;
    Chunk<T> xq[VPT], rq[VPT], yq[VPT], gq[VPT];
    float d[VPT][8], s1[1] = {0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (c >= S.chunks || !live) continue;
      if (A.dres) rq[v].load(rr, c * 8);
      if (JOIN) yq[v].load(ry_, c * 8);
      if (full) gq[v].load(rg, c * 8);
      if (next) {
        Chunk<T> dq;
        dq.load(rd, c * 8);
        xq[v].load(rx, c * 8);
        float ga[8], x[8];
        load_f8(gamma_n, c * 8, ga);
        xq[v].get(x);
        dq.get(d[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xn = x[i] * rn;
          sn[v][i] = fmaf(d[v][i], xn, sn[v][i]);
          d[v][i] *= S.offset + ga[i];
          s1[0] = fmaf(d[v][i], xn, s1[0]);
        }
      }
    }
    if (!__syncthreads_and(arrived)) {  // the stage has been read, or a copy is overdue
      ring.abandon();
      return;
    }
    if (threadIdx.x == 0) ring.issue(it + S.stages);
    float m = 0.f;
    if (next) {
      group_sum<1>(s1, S.group, sh.red, turn);
      m = s1[0] * S.inv_h * rn * rn;
    }
    float s2[2] = {0.f, 0.f};  // sum of b yn; of d u (the token gate's gradient)
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (c >= S.chunks || !live) continue;
      if (next) {
        float x[8];
        xq[v].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[v][i] = rn * d[v][i] - x[i] * m;
      }
      if (A.dres) {
        float f[8];
        rq[v].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[v][i] = next ? d[v][i] + f[i] : f[i];
      }
      Chunk<T>::store(A.dx, row + c * 8, d[v]);
      if (JOIN) {
        float y[8], ga[8], gt[8], dg[8];
        yq[v].get(y);
        load_f8(A.gamma, c * 8, ga);
        if (full) gq[v].get(gt);
        if (CHANNEL) load_f8((const float*)A.gate, c * 8, gt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float yn = y[i] * ry, gp = S.offset + ga[i], sd = S.scale * d[v][i];
          const float vv = sd * (full || CHANNEL ? gt[i] : tok);
          dg[i] = sd * yn * gp;
          sp[v][i] = fmaf(vv, yn, sp[v][i]);
          if (CHANNEL) sg[v][i] += dg[i];
          s2[1] += dg[i];
          d[v][i] = vv * gp;  // b
          s2[0] = fmaf(d[v][i], yn, s2[0]);
        }
        if (full) Chunk<T>::store(A.dgate, row + c * 8, dg);
      }
    }
    if (JOIN) {
      group_sum<2>(s2, S.group, sh.red, turn);
      const float my = s2[0] * S.inv_h * ry * ry;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = g + v * S.group;
        if (c >= S.chunks || !live) continue;
        float y[8];
        yq[v].get(y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = ry * d[v][i] - y[i] * my;
        Chunk<T>::store(A.dy, row + c * 8, y);
      }
      if (live && g == 0 && S.gate == MOE_GATE_TOKEN) ((float*)A.dgate)[t] = s2[1];
    }
  }

  // The CTA's column sums: its groups' sums are added in order through shared memory (the ring,
  // which no copy uses any more), then leave as a partial row, or as the result of a lone CTA.
  auto leave = [&](float (&s)[VPT][8], int kind) {
    float* to = gridDim.x == 1 ? outs.p[kind]
                               : A.ws + ((int64_t)blockIdx.x * kinds + kind) * S.H;
    if (S.per > 1) {
      float* all = (float*)smem;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = g + v * S.group;
        if (c < S.chunks) Chunk<float>::store(all + (int64_t)local * S.H, c * 8, s[v]);
      }
      __syncthreads();
      for (int c = threadIdx.x; c < S.H; c += blockDim.x) {
        float sum = 0.f;
        for (int l = 0; l < S.per; ++l) sum += all[l * S.H + c];
        to[c] = sum;
      }
    } else {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = g + v * S.group;
        if (c < S.chunks) {
#pragma unroll
          for (int i = 0; i < 8; ++i) to[c * 8 + i] = s[v][i];
        }
      }
    }
  };
  int kind = 0;
  if constexpr (JOIN) leave(sp, kind++);
  if (next) leave(sn, kind++);
  if constexpr (CHANNEL) leave(sg, kind++);
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

// Threads a row: one chunk of 8 elements each up to 256 chunks, then 2, 4, 8, so that a CTA has at
// most 512 threads; short rows share a CTA of 256.
static int vec_of(int H) {
  const int chunks = H / 8;
  return chunks <= 256 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8;
}
static Shape shape_of(const moe_block_t& c) {
  Shape s{};
  s.T = c.T;
  s.H = c.H;
  s.chunks = c.H / 8;
  s.group = ceil_div(ceil_div(s.chunks, vec_of(c.H)), 32) * 32;
  s.per = std::min(c.T, std::max(1, 256 / s.group));
  s.units = ceil_div(c.T, s.per);
  s.scale = c.scale;
  s.offset = c.offset;
  s.eps = c.eps;
  s.inv_h = 1.0f / (float)c.H;
  s.gate = c.gate_kind;
  return s;
}

// Partial rows at most: the backward kernels' CTAs.
constexpr int kMaxCtas = 4;  // an SM
static int max_blocks(const Shape& s) { return std::min(s.units, num_sms() * kMaxCtas); }

// Fills in the ring: as many of the row tensors as fit, and as many stages as the budget of an
// SM's resident CTAs allows. Returns the CTA's dynamic shared memory.
static size_t plan_ring(Shape& s, size_t es, int ctas) {
  const size_t one = (size_t)s.per * s.H * es;
  s.ringed = std::min<int>(s.n_in, (int)(kMaxRing / one));
  const size_t stage = one * s.ringed;
  s.stages = 1;
  if (s.ringed)
    s.stages = (int)std::min<size_t>(kMaxStages, std::max<size_t>(1, kRingBudget / ctas / stage));
  return stage * s.stages;
}

template <typename... KArgs, typename... Args>
static moe_status_t run(void (*kern)(KArgs...), Shape& S, size_t es, size_t least, int max_ctas,
                        int& blocks, cudaStream_t s, Args&&... args) {
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
  size_t smem = std::max(plan_ring(S, es, ctas), least);
  ctas = std::max(1, std::min<int>(ctas, (int)(220 * 1024 / (smem + 1024))));
  blocks = std::min(S.units, num_sms() * ctas);
  return launch_k(kern, dim3(blocks), dim3(threads), smem, s, (const Shape&)S,
                  std::forward<Args>(args)...);
}

template <bool JOIN>
static moe_status_t forward(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  Shape S = shape_of(c);
  if (JOIN) S.in[S.n_in++] = a.y;
  S.in[S.n_in++] = a.x;
  if (JOIN && c.gate_kind == MOE_GATE_FULL) S.in[S.n_in++] = a.gate;
  int blocks = 0;
  auto go = [&](auto kern) { return run(kern, S, dtype_size(c.dtype), 0, 8, blocks, s, a); };
  using bf = __nv_bfloat16;
  const int v = vec_of(c.H);
  if (c.dtype == MOE_BF16)
    return v == 1   ? go(forward_kernel<bf, 1, JOIN>)
           : v == 2 ? go(forward_kernel<bf, 2, JOIN>)
           : v == 4 ? go(forward_kernel<bf, 4, JOIN>) : go(forward_kernel<bf, 8, JOIN>);
  return v == 1   ? go(forward_kernel<float, 1, JOIN>)
         : v == 2 ? go(forward_kernel<float, 2, JOIN>)
         : v == 4 ? go(forward_kernel<float, 4, JOIN>) : go(forward_kernel<float, 8, JOIN>);
}

template <bool JOIN, bool CHANNEL>
static moe_status_t backward(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  Shape S = shape_of(c);
  const bool next = !JOIN || a.gamma_next;
  if (next) {
    S.in[S.n_in++] = a.dh;
    S.in[S.n_in++] = JOIN ? a.out_in : a.x;
  }
  if (a.dres) S.in[S.n_in++] = a.dres;
  if (JOIN) S.in[S.n_in++] = a.y;
  if (JOIN && c.gate_kind == MOE_GATE_FULL) S.in[S.n_in++] = a.gate;
  Outs outs{};
  int kinds = 0;
  outs.p[kinds++] = a.dgamma;
  if (JOIN && next) outs.p[kinds++] = a.dgamma_next;
  if (CHANNEL) outs.p[kinds++] = (float*)a.dgate;
  // the CTA's groups meet in shared memory at the end
  const size_t least = S.per > 1 ? (size_t)S.per * S.H * sizeof(float) : 0;
  int blocks = 0;
  auto go = [&](auto kern) {
    return run(kern, S, dtype_size(c.dtype), least, kMaxCtas, blocks, s, a, kinds, outs);
  };
  using bf = __nv_bfloat16;
  const int v = vec_of(c.H);
  moe_status_t st;
  if (c.dtype == MOE_BF16)
    st = v == 1   ? go(backward_kernel<bf, 1, JOIN, CHANNEL>)
         : v == 2 ? go(backward_kernel<bf, 2, JOIN, CHANNEL>)
         : v == 4 ? go(backward_kernel<bf, 4, JOIN, CHANNEL>)
                  : go(backward_kernel<bf, 8, JOIN, CHANNEL>);
  else
    st = v == 1   ? go(backward_kernel<float, 1, JOIN, CHANNEL>)
         : v == 2 ? go(backward_kernel<float, 2, JOIN, CHANNEL>)
         : v == 4 ? go(backward_kernel<float, 4, JOIN, CHANNEL>)
                  : go(backward_kernel<float, 8, JOIN, CHANNEL>);
  if (st != MOE_OK || blocks == 1) return st;
  return launch_k(column_sum_kernel, dim3(ceil_div(kinds * c.H, 32)), dim3(1024), 0, s,
                  (const float*)a.ws, blocks, kinds, c.H, outs);
}

}  // namespace bnorm

using namespace bnorm;

size_t block_norm_ws_bytes(const moe_block_t& c) {
  return (size_t)max_blocks(shape_of(c)) * 3 * c.H * sizeof(float);
}

int block_norm_status_read(int reset) {
  int v = 0;
  cudaMemcpyFromSymbol(&v, bnorm::g_status, sizeof(int));
  if (reset) {
    int z = 0;
    cudaMemcpyToSymbol(bnorm::g_status, &z, sizeof(int));
  }
  return v;
}

moe_status_t launch_block_norm(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  return forward<false>(c, a, s);
}
moe_status_t launch_block_join(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s) {
  return forward<true>(c, a, s);
}
moe_status_t launch_block_norm_backward(const moe_block_t& c, const BlockNormArgs& a,
                                        cudaStream_t s) {
  return backward<false, false>(c, a, s);
}
moe_status_t launch_block_join_backward(const moe_block_t& c, const BlockNormArgs& a,
                                        cudaStream_t s) {
  return c.gate_kind == MOE_GATE_CHANNEL ? backward<true, true>(c, a, s)
                                         : backward<true, false>(c, a, s);
}

}  // namespace moe
