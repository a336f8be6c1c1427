// balance.cu — the router's balance and z losses with the experts' counts, and their gradient
// (moe_balance_loss, moe_balance_loss_backward).
//
// For a token with logits z: l = log sum_e exp z_e; p = softmax z, or sigma(z) / sum sigma(z).
//   balance = 1/S' sum_s sum_e E c_se / (k n_s) P_se,  P_se = 1/n_s sum_t p_te;   z loss = 1/N sum_t l_t^2
//   gradient, with g_e = E c_se / (k n_s) / (n_s S'):
//     dz_e = d0 p_e (g_e - sum g p) [1 - sigma(z_e), sigmoid routing] + d1 2 l / N softmax(z)_e
// The logits are read once each way, so HBM would bound both directions, but a batch's logits are a few
// megabytes: launches and the latency of one token's sums count as much. A group of G lanes (a power
// of two) takes a token, lane i holding experts i, i + G, ...; a CTA takes a chunk of consecutive tokens,
// sequence by sequence, and leaves partial sums in slot chunk + s, a place of its own for every pair of a
// chunk and a sequence that meet, since both only grow along the tokens. A second kernel adds a
// sequence's slots in order. Counts are integers, everything else is added in a fixed order.
#include "stack.cuh"
#include "train.cuh"

namespace moe {
namespace balance {

__device__ int g_status;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxE = 512;

struct Args {
  const float *logits, *bias;
  const int32_t *ids, *offsets;
  const uint8_t* mask;
  int T, E, k, slots, S, group;  // group: lanes of a token
  int per_chunk;                 // tokens of a CTA
  int sigmoid;
  // partial sums: P [slots][E], counts [slots][E], then live tokens and sums of l^2 [slots]
  float* part_p;
  int32_t* part_c;
  int32_t* part_n;
  float* part_z;
};

// The run of tokens of one sequence that holds token t of a chunk that ends before `end`: its sequence
// and its end. s < 0: tokens of no sequence.
struct Run {
  int s, end;
};
__device__ __forceinline__ Run run_of(const Args& A, int t, int end) {
  if (!A.offsets) return {0, end};
  int lo = 0, hi = A.S + 1;  // the first offset beyond t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(A.offsets + mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  if (lo == 0) return {-1, max(t + 1, min(end, __ldg(A.offsets)))};
  if (lo == A.S + 1) return {-1, end};
  return {lo - 1, max(t + 1, min(end, __ldg(A.offsets + lo)))};
}

__device__ __forceinline__ float group_max(float v, int group) {
  for (int off = group >> 1; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float group_add(float v, int group) {
  for (int off = group >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A token's probabilities from its logits, in the lanes of its group.
template <int N>
struct Token {
  float p[N], soft[N], slope[N];  // p; softmax; 1 - sigma(z), or 1
  float lse;
  // z: -inf beyond the experts. Sigmoids are taken relative to e^max where all logits are negative: p
  // stays right where every sigmoid underflows.
  __device__ __forceinline__ void set(const float (&z)[N], int group, bool sigmoid) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, z[i]);
    m = group_max(m, group);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      soft[i] = expf(z[i] - m);
      sum += soft[i];
    }
    float total = 0.f;
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = expf(-fabsf(z[i])), d = 1.f / (1.f + x);
        p[i] = m < 0.f ? soft[i] * d : z[i] >= 0.f ? d : x * d;
        slope[i] = z[i] >= 0.f ? x * d : d;
        total += p[i];
      }
    }
    sum = group_add(sum, group);
    lse = m + logf(sum);
    const float inv = 1.f / sum;
#pragma unroll
    for (int i = 0; i < N; ++i) soft[i] *= inv;
    if (sigmoid) {
      const float norm = 1.f / group_add(total, group);
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] *= norm;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p[i] = soft[i];
        slope[i] = 1.f;
      }
    }
  }
};

template <int N>
__device__ __forceinline__ void load_logits(const Args& A, int64_t t, bool live, int gl,
                                            float (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = gl + i * A.group;
    z[i] = live && e < A.E ? __ldg(A.logits + t * A.E + e) : -INFINITY;
  }
}

// Sums over the chunks' tokens.
template <int N>
__global__ void __launch_bounds__(kThreads) partial_kernel(const __grid_constant__ Args A,
                                                           int* arrived) {
  extern __shared__ float sums[];  // [warps][E]
  __shared__ int cnt[kMaxE];
  __shared__ float zs[kWarps];
  __shared__ int ns[kWarps];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *arrived = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = A.group, gl = lane & (G - 1), at_once = kThreads / G, sub = threadIdx.x / G;
  const int t0 = blockIdx.x * A.per_chunk, t1 = min(A.T, t0 + A.per_chunk);
  float bias[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = gl + i * G;
    bias[i] = A.bias && e < A.E ? __ldg(A.bias + e) : 0.f;
  }
  for (int t = t0; t < t1;) {
    const Run r = run_of(A, t, t1);
    if (r.s < 0) {
      t = r.end;
      continue;
    }
    for (int e = threadIdx.x; e < A.E; e += kThreads) cnt[e] = 0;
    __syncthreads();
    float acc[N], z2 = 0.f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    float z[N];
    bool live = t + sub < r.end && (!A.mask || A.mask[t + sub]);
    load_logits<N>(A, t + sub, live, gl, z);
    for (int b = t; b < r.end; b += at_once) {
      const int64_t mine = (int64_t)b + sub, then = mine + at_once;
      float zn[N];
      const bool next = then < r.end && (!A.mask || A.mask[then]);
      load_logits<N>(A, then, next, gl, zn);
      if (live) {
        for (int j = gl; j < A.k; j += G) {
          const int id = __ldg(A.ids + mine * A.slots + j);
          if (id >= 0 && id < A.E) atomicAdd(&cnt[id], 1);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] += bias[i];
      Token<N> k;
      k.set(z, G, A.sigmoid);
      if (live) {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += k.p[i];
        z2 += k.lse * k.lse;
        ++n;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = zn[i];
      live = next;
    }
    // over a warp's tokens, then over the warps, in order
#pragma unroll
    for (int i = 0; i < N; ++i)
      for (int off = G; off < 32; off <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
    for (int off = G; off < 32; off <<= 1) {
      z2 += __shfl_xor_sync(0xffffffffu, z2, off);
      n += __shfl_xor_sync(0xffffffffu, n, off);
    }
    if (lane < G) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (gl + i * G < A.E) sums[warp * A.E + gl + i * G] = acc[i];
    }
    if (lane == 0) {
      zs[warp] = z2;
      ns[warp] = n;
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + r.s;
    for (int e = threadIdx.x; e < A.E; e += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w * A.E + e];
      A.part_p[slot * A.E + e] = s;
      A.part_c[slot * A.E + e] = cnt[e];
    }
    if (threadIdx.x == 0) {
      float s = 0.f;
      int c = 0;
      for (int w = 0; w < kWarps; ++w) {
        s += zs[w];
        c += ns[w];
      }
      A.part_z[slot] = s;
      A.part_n[slot] = c;
    }
    __syncthreads();
    t = r.end;
  }
}

struct Sums {  // outputs, and what the sequences leave for the last CTA
  float *losses, *prob;
  int32_t *counts, *tokens, *totals;
  float *loss_part, *z_part;  // [S][column blocks], [S]
  int* arrived;
};

// A CTA adds up 32 experts of a sequence; the one that ends last adds up the losses.
__global__ void __launch_bounds__(256) sequence_kernel(const __grid_constant__ Args A,
                                                       const __grid_constant__ Sums B) {
  __shared__ float sp[8][33], sz[8];
  __shared__ int sc[8][33], sn[8];
  __shared__ bool last;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = (A.E + 31) / 32;
  const int s = blockIdx.x / blocks, eb = blockIdx.x % blocks, e = eb * 32 + lane;
  int a = A.offsets ? __ldg(A.offsets + s) : 0, b = A.offsets ? __ldg(A.offsets + s + 1) : A.T;
  if (a < 0 || b < a || b > A.T) {
    if (threadIdx.x == 0) atomicExch(&g_status, kStatusBadOffsets);
    a = min(max(a, 0), A.T);
    b = min(max(b, a), A.T);
  }
  const int64_t first = a / A.per_chunk + s;
  const int chunks = b > a ? (b - 1) / A.per_chunk - a / A.per_chunk + 1 : 0;
  float p = 0.f, z = 0.f;
  int c = 0, n = 0;
#pragma unroll 4
  for (int i = warp; i < chunks; i += 8) {
    const int64_t slot = first + i;
    if (e < A.E) {
      p += A.part_p[slot * A.E + e];
      c += A.part_c[slot * A.E + e];
    }
  }
  for (int i = threadIdx.x; i < chunks; i += 256) {
    n += A.part_n[first + i];
    z += A.part_z[first + i];
  }
  sp[warp][lane] = p;
  sc[warp][lane] = c;
  z = warp_total(z);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    sz[warp] = z;
    sn[warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    p = z = 0.f;
    c = n = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      p += sp[w][lane];
      c += sc[w][lane];
      z += sz[w];
      n += sn[w];
    }
    const float inv = n ? 1.f / (float)n : 0.f;
    p *= inv;
    if (e < A.E) {
      B.prob[(int64_t)s * A.E + e] = p;
      B.counts[(int64_t)s * A.E + e] = c;
    }
    const float loss = warp_total(e < A.E ? (float)c * ((float)A.E / (float)A.k) * inv * p : 0.f);
    if (lane == 0) {
      B.loss_part[blockIdx.x] = loss;
      if (eb == 0) {
        B.z_part[s] = z;
        B.tokens[s] = n;
      }
      __threadfence();
      last = atomicAdd(B.arrived, 1) == (int)gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float loss = 0.f;
  int some = 0;
  z = 0.f;
  n = 0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += 256) loss += __ldcg(B.loss_part + i);
  for (int i = threadIdx.x; i < A.S; i += 256) {
    const int m = __ldcg(B.tokens + i);
    z += __ldcg(B.z_part + i);
    n += m;
    some += m > 0;
  }
  loss = warp_total(loss);
  z = warp_total(z);
  n = __reduce_add_sync(0xffffffffu, n);
  some = __reduce_add_sync(0xffffffffu, some);
  if (lane == 0) {
    sp[warp][0] = loss;
    sp[warp][1] = z;
    sc[warp][0] = n;
    sc[warp][1] = some;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    loss = z = 0.f;
    n = some = 0;
    for (int w = 0; w < 8; ++w) {
      loss += sp[w][0];
      z += sp[w][1];
      n += sc[w][0];
      some += sc[w][1];
    }
    B.losses[0] = some ? loss / (float)some : 0.f;
    B.losses[1] = n ? z / (float)n : 0.f;
    B.totals[0] = some;
    B.totals[1] = n;
  }
}

// The gradient: the same walk over the tokens, a sequence's weights in registers.
template <int N>
__global__ void __launch_bounds__(256) backward_kernel(const __grid_constant__ Args A,
                                                       const float* __restrict__ dlosses,
                                                       const int32_t* __restrict__ counts,
                                                       const int32_t* __restrict__ tokens,
                                                       const int32_t* __restrict__ totals, int add,
                                                       float* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int G = A.group, gl = lane & (G - 1), at_once = 256 / G, sub = threadIdx.x / G;
  const int t0 = blockIdx.x * A.per_chunk, t1 = min(A.T, t0 + A.per_chunk);
  const int some = __ldg(totals), all = __ldg(totals + 1);
  const float d0 = __ldg(dlosses), d1 = __ldg(dlosses + 1) * 2.f / (float)max(all, 1);
  float bias[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = gl + i * G;
    bias[i] = A.bias && e < A.E ? __ldg(A.bias + e) : 0.f;
  }
  for (int t = t0; t < t1;) {
    const Run r = run_of(A, t, t1);
    float g[N];
    if (r.s >= 0) {
      const float n = (float)max(__ldg(tokens + r.s), 1);
      const float f = d0 * ((float)A.E / (float)A.k) / (n * n * (float)max(some, 1));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = gl + i * G;
        g[i] = e < A.E ? f * (float)__ldg(counts + (int64_t)r.s * A.E + e) : 0.f;
      }
    }
    for (int b = t; b < r.end; b += at_once) {
      const int64_t mine = (int64_t)b + sub;
      const bool in = mine < r.end, live = in && r.s >= 0 && (!A.mask || A.mask[mine]);
      float z[N], d[N];
      load_logits<N>(A, mine, live, gl, z);
      if (add) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          d[i] = live && gl + i * G < A.E ? dlogits[mine * A.E + gl + i * G] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] += bias[i];
      Token<N> k;
      k.set(z, G, A.sigmoid);
      float dot = 0.f;
      if (r.s >= 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) dot = fmaf(g[i], k.p[i], dot);
      }
      dot = group_add(dot, G);
      const float dl = d1 * k.lse;
      if (!in || (add && !live)) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (gl + i * G >= A.E) continue;
        float v = live ? fmaf(k.p[i] * k.slope[i], g[i] - dot, dl * k.soft[i]) : 0.f;
        if (add) v += d[i];
        dlogits[mine * A.E + gl + i * G] = v;
      }
    }
    t = r.end;
  }
}

// Lanes of a token and experts a lane.
static int group_of(int E) {
  int g = 1;
  while (g < 32 && g < E) g <<= 1;
  return g;
}
static Args args_of(const moe_balance_t& c, const float* logits, int ctas, int threads) {
  Args A{};
  A.logits = logits;
  A.bias = c.mode == MOE_ROUTE_SOFTMAX ? c.logit_bias : nullptr;
  A.offsets = c.offsets;
  A.mask = c.mask;
  A.T = c.T;
  A.E = c.E;
  A.k = c.k;
  A.slots = c.k + c.n_shared;
  A.S = c.offsets ? c.S : 1;
  A.group = group_of(c.E);
  A.sigmoid = c.mode == MOE_ROUTE_SIGMOID_GROUPED;
  // every thread's group has a token where there are enough
  A.per_chunk = std::max(threads / A.group, ceil_div(c.T, ctas));
  return A;
}
static int forward_ctas() { return num_sms() * 2; }
struct Layout {
  size_t p, c, n, z, loss, zs, arrived, total;
};
static Layout layout(const moe_balance_t& c) {
  const Args A = args_of(c, nullptr, forward_ctas(), kThreads);
  const size_t slots = (size_t)ceil_div(A.T, A.per_chunk) + A.S;
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t v = at;
    at += align_up(bytes, 256);
    return v;
  };
  l.p = take(slots * A.E * 4);
  l.c = take(slots * A.E * 4);
  l.n = take(slots * 4);
  l.z = take(slots * 4);
  l.loss = take((size_t)A.S * ceil_div(A.E, 32) * 4);
  l.zs = take((size_t)A.S * 4);
  l.arrived = take(4);
  l.total = at;
  return l;
}

#define BALANCE_PICK(name)                    \
  (c.E <= 32    ? go(name<1>)                 \
   : c.E <= 64  ? go(name<2>)                 \
   : c.E <= 128 ? go(name<4>)                 \
   : c.E <= 256 ? go(name<8>)                 \
                : go(name<16>))

}  // namespace balance

using namespace balance;

size_t balance_ws_bytes(const moe_balance_t& c) { return layout(c).total; }

moe_status_t launch_balance(const moe_balance_t& c, const float* logits, const int32_t* ids,
                            float* losses, int32_t* counts, int32_t* tokens, float* prob,
                            int32_t* totals, void* ws, cudaStream_t s) {
  Args A = args_of(c, logits, forward_ctas(), kThreads);
  const Layout l = layout(c);
  uint8_t* w = (uint8_t*)ws;
  A.ids = ids;
  A.part_p = (float*)(w + l.p);
  A.part_c = (int32_t*)(w + l.c);
  A.part_n = (int32_t*)(w + l.n);
  A.part_z = (float*)(w + l.z);
  Sums B{losses, prob, counts, tokens, totals, (float*)(w + l.loss), (float*)(w + l.zs), (int*)(w + l.arrived)};
  auto go = [&](auto kern) {
    return launch_k(kern, dim3(ceil_div(c.T, A.per_chunk)), dim3(kThreads),
                    (size_t)kWarps * c.E * sizeof(float), s, (const Args&)A, B.arrived);
  };
  const moe_status_t st = BALANCE_PICK(partial_kernel);
  if (st != MOE_OK) return st;
  return launch_k(sequence_kernel, dim3(A.S * ceil_div(c.E, 32)), dim3(256), 0, s, (const Args&)A, (const Sums&)B);
}

moe_status_t launch_balance_backward(const moe_balance_t& c, const float* dlosses,
                                     const float* logits, const int32_t* counts,
                                     const int32_t* tokens, const int32_t* totals, int accumulate,
                                     float* dlogits, cudaStream_t s) {
  const Args A = args_of(c, logits, num_sms() * 4, 256);
  auto go = [&](auto kern) {
    return launch_k(kern, dim3(ceil_div(c.T, A.per_chunk)), dim3(256), 0, s, A, dlosses, counts, tokens,
                    totals, accumulate, dlogits);
  };
  return BALANCE_PICK(backward_kernel);
}

int balance_status_read(int reset) {
  int v = 0;
  cudaMemcpyFromSymbol(&v, g_status, sizeof(int));
  if (reset) {
    int z = 0;
    cudaMemcpyToSymbol(g_status, &z, sizeof(int));
  }
  return v;
}

}  // namespace moe
