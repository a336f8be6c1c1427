// balance.cu — the router's balance and z losses with the experts' counts, and their gradient
// (moe_balance_loss, moe_balance_loss_backward).
//
// For a token with logits z: l = log sum_e exp z_e; p = softmax z, or sigma(z) / sum sigma(z).
//   balance = 1/S' sum_s sum_e E c_se / (k n_s) P_se,  P_se = 1/n_s sum_t p_te;   z loss = 1/N sum_t l_t^2
//   gradient, with g_e = E c_se / (k n_s) / (n_s S'):
//     dz_e = d0 p_e (g_e - sum g p) [1 - sigma(z_e), sigmoid routing] + d1 2 l / N softmax(z)_e
// The logits are read once each way, so HBM would bound both directions, but a batch's logits are a few
// megabytes: instructions, launches and latencies count more. A group of G lanes (a power of two) takes a
// token, up to 16 experts a lane: with a whole warp a token, the shuffles of its sums took most of the time.
// A CTA takes a chunk of consecutive tokens, sequence by sequence, and leaves partial sums in slot chunk + s, a
// place of its own for every pair of a chunk and a sequence that meet, since both only grow along the
// tokens. A second kernel adds a sequence's slots in order. Counts are integers, everything else is
// added in a fixed order.
// Measured, from a cold L2: 32768 tokens of 128 experts, softmax, 9 us, 7 for the second kernel, 9 backward (16, 8
// and 20 with a warp a token; the bytes need 2.5 each way); 8191 of 256, sigmoids, in 13 sequences 10, 6 and 9.
// With the logits in L2 22 and 24 us in all; added to a gradient that is there 10 and 5 more.
#include "stack.cuh"
#include "train.cuh"

namespace moe {
namespace balance {

__device__ int g_status;

constexpr int kThreads = 512, kWarps = kThreads / 32;  // forward
constexpr int kBackThreads = 256;
constexpr int kNear = 2048;  // offsets that are looked up in shared memory

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
struct Offsets {
  int32_t near[kNear];
  // Called by all threads of the CTA.
  __device__ __forceinline__ void fetch(const Args& A) {
    if (!A.offsets || A.S >= kNear) return;
    for (int i = threadIdx.x; i <= A.S; i += blockDim.x) near[i] = __ldg(A.offsets + i);
    __syncthreads();
  }
  __device__ __forceinline__ Run run(const Args& A, int t, int end) const {
    if (!A.offsets) return {0, end};
    const int32_t* off = A.S < kNear ? near : A.offsets;
    int lo = 0, hi = A.S + 1;  // the first offset beyond t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (off[mid] <= t) lo = mid + 1;
      else hi = mid;
    }
    if (lo > A.S) return {-1, end};
    return {lo - 1, max(t + 1, min(end, off[lo]))};
  }
};

__device__ __forceinline__ float group_max(float v, int group) {
  for (int off = group >> 1; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float group_add(float v, int group) {
  for (int off = group >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The experts of a lane: pieces of four consecutive ones, or (VEC false: E is no multiple of 4) single
// ones, of its group in turn. Beyond the last expert e >= E.
template <int N, bool VEC>
__device__ __forceinline__ int expert(int i, int gl, int G) {
  return VEC ? (i / 4 * G + gl) * 4 + i % 4 : gl + i * G;
}
template <int N, bool VEC>
__device__ __forceinline__ void load_lane(const float* row, bool in, int E, int gl, int G, float beyond,
                                          float (&v)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const int e = expert<N, VEC>(i, gl, G);
      float4 q = make_float4(beyond, beyond, beyond, beyond);
      if (in && e < E) q = __ldg((const float4*)(row + e));
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = expert<N, VEC>(i, gl, G);
      v[i] = in && e < E ? __ldg(row + e) : beyond;
    }
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A token's probabilities from its logits, in the lanes of its group.
template <int N, bool SIGMOID>
struct Token {
  float p[N];
  float soft[SIGMOID ? N : 1], slope[SIGMOID ? N : 1];  // softmax; 1 - sigma(z)
  float lse;
  // z: -inf beyond the experts. Sigmoids are taken relative to e^max where all logits are negative: p
  // stays right where every sigmoid underflows.
  __device__ __forceinline__ void set(const float (&z)[N], int group) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, z[i]);
    m = group_max(m, group);
    // exponentials of base 2: off by 2 steps, and by half a step for every unit of z - m
    constexpr float kLog2e = 1.4426950408889634f;
    const float shift = -m * kLog2e;
    float sum = 0.f, total = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = exp2_fast(fmaf(z[i], kLog2e, shift));
      sum += p[i];
    }
    if constexpr (SIGMOID) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // an accurate exponential: a rounded product of z and log2(e) alone puts x off by up to 16 half steps at
        // z = -20, 58 at -60 (above, the error is that of the difference to the largest, which any form has).
        // The reciprocal is off by one step whatever z. Both directions, 8191 tokens of 256 experts, 23.2 us with the
        // approximate exponential, 24.1 so, 26.3 with a true division too.
        const float x = expf(-fabsf(z[i])), d = reciprocal_fast(1.f + x);
        soft[i] = p[i];
        p[i] = m < 0.f ? p[i] * d : z[i] >= 0.f ? d : x * d;
        slope[i] = z[i] >= 0.f ? x * d : d;
        total += p[i];
      }
      total = group_add(total, group);
    }
    sum = group_add(sum, group);
    lse = m + logf(sum);
    const float inv = 1.f / sum, norm = SIGMOID ? 1.f / total : inv;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] *= norm;
      if constexpr (SIGMOID) soft[i] *= inv;
    }
  }
};

// The tokens of a tile, one a group, and whether they take part; asked for a tile ahead.
template <int N, bool VEC>
struct Tile {
  float z[N];
  bool live;
  __device__ __forceinline__ void ask(const Args& A, int64_t t, int64_t end, int gl) {
    live = t < end;
    load_lane<N, VEC>(A.logits + t * A.E, live, A.E, gl, A.group, -INFINITY, z);
    if (live && A.mask) live = A.mask[t];
  }
  __device__ __forceinline__ void add_bias(const Args& A, int gl) {
    if (!A.bias) return;
    float bias[N];
    load_lane<N, VEC>(A.bias, true, A.E, gl, A.group, 0.f, bias);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] += bias[i];
  }
};

// Sums over the chunks' tokens. All that a chunk's first tile needs is asked for before anything is waited
// for; a tile's probabilities are computed once, and added to every sequence that it meets.
template <int N, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, 2) partial_kernel(const __grid_constant__ Args A,
                                                              int* arrived) {
  __shared__ __align__(16) float sums[kThreads * N];  // [groups][lanes * N]: every token group's sums
  __shared__ float part[kThreads];                    // [parts][lanes * N]: N groups' each
  __shared__ int cnt[512];
  __shared__ float zs[kThreads];  // of the groups
  __shared__ int ns[kThreads];
  __shared__ Offsets off;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = A.group, gl = lane & (G - 1), groups = kThreads / G, sub = threadIdx.x / G;
  const int t0 = blockIdx.x * A.per_chunk, t1 = min(A.T, t0 + A.per_chunk);
  Tile<N, VEC> tile;
  tile.ask(A, (int64_t)t0 + sub, t1, gl);
  // one slot of the chunk a thread; the few beyond are read when they are counted
  const int slots = (t1 - t0) * A.slots;
  auto id_of = [&](int i, int t) {  // slot i of the chunk, of token t; -1: not counted
    if (i >= slots || i - (t - t0) * A.slots >= A.k) return -1;
    const int id = __ldg(A.ids + (int64_t)t0 * A.slots + i);
    return (!A.mask || A.mask[t]) && id < A.E ? id : -1;
  };
  const int my_token = t0 + (int)(threadIdx.x / (unsigned)A.slots), my_id = id_of(threadIdx.x, my_token);
  if (blockIdx.x == 0 && threadIdx.x == 0) *arrived = 0;
  off.fetch(A);
  int start = t0;
  Run r = off.run(A, t0, t1);
  float acc[N], z2 = 0.f;
  int n = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;

  auto flush = [&]() {  // the sums of run r, which began at `start`, into its slot
    for (int e = threadIdx.x; e < A.E; e += kThreads) cnt[e] = 0;
    // all groups' sums through shared memory, first over N groups, then over those, in order
    const int width = G * N;
    float* row = sums + sub * width;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *(float4*)(row + expert<N, VEC>(i, gl, G)) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) row[expert<N, VEC>(i, gl, G)] = acc[i];
    }
    if (gl == 0) zs[sub] = z2;
    if (gl == 0) ns[sub] = n;
    __syncthreads();
    const int column = threadIdx.x % width, first = threadIdx.x / width * N;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += sums[(first + i) * width + column];
    part[threadIdx.x] = s;
    if (my_id >= 0 && my_token >= start && my_token < r.end) atomicAdd(&cnt[my_id], 1);
    for (int i = threadIdx.x + kThreads; i < slots; i += kThreads) {
      const int t = t0 + i / A.slots;
      if (t < start || t >= r.end) continue;
      const int id = id_of(i, t);
      if (id >= 0) atomicAdd(&cnt[id], 1);
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + r.s;
    for (int e = threadIdx.x; e < A.E; e += kThreads) {
      s = 0.f;
      for (int w = e; w < kThreads; w += width) s += part[w];
      A.part_p[slot * A.E + e] = s;
      A.part_c[slot * A.E + e] = cnt[e];
    }
    if (warp == kWarps - 1) {
      s = 0.f;
      int c = 0;
      for (int i = lane; i < groups; i += 32) {
        s += zs[i];
        c += ns[i];
      }
      s = warp_total(s);
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) {
        A.part_z[slot] = s;
        A.part_n[slot] = c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    z2 = 0.f;
    n = 0;
  };

  for (int b = t0; b < t1; b += groups) {
    const int mine = b + sub;
    const bool live = tile.live;
    tile.add_bias(A, gl);
    Token<N, SIGMOID> k;
    k.set(tile.z, G);
    tile.ask(A, (int64_t)mine + groups, t1, gl);
    for (;;) {
      if (r.s >= 0 && live && mine >= start && mine < r.end) {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += k.p[i];
        z2 += k.lse * k.lse;
        ++n;
      }
      if (r.end - groups > b) break;  // the run goes on behind the tile
      if (r.s >= 0) flush();
      if (r.end >= t1) break;
      start = r.end;
      r = off.run(A, start, t1);
    }
  }
}

struct Sums {  // outputs, and what the sequences leave for the last CTA
  float *losses, *prob;
  int32_t *counts, *tokens, *totals;
  float *loss_part, *z_part;  // [S][E / 8 rounded up], [S]
  int* arrived;
};

// Sums over a CTA's threads, in thread 0.
template <int WARPS>
struct BlockSum {
  float f[2][WARPS];
  int i[2][WARPS];
  __device__ __forceinline__ void add(float& a, float& b, int& c, int& d) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = warp_total(a);
    b = warp_total(b);
    c = __reduce_add_sync(0xffffffffu, c);
    d = __reduce_add_sync(0xffffffffu, d);
    if (lane == 0) {
      f[0][warp] = a;
      f[1][warp] = b;
      i[0][warp] = c;
      i[1][warp] = d;
    }
    __syncthreads();
    if (warp == 0) {
      a = warp_total(lane < WARPS ? f[0][lane] : 0.f);
      b = warp_total(lane < WARPS ? f[1][lane] : 0.f);
      c = __reduce_add_sync(0xffffffffu, lane < WARPS ? i[0][lane] : 0);
      d = __reduce_add_sync(0xffffffffu, lane < WARPS ? i[1][lane] : 0);
    }
    __syncthreads();
  }
};

// A CTA adds up 8 experts of a sequence, its threads slots side by side; the one that ends last adds up
// the losses. WARPS: many for few sequences, which have many slots.
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32) sequence_kernel(const __grid_constant__ Args A,
                                                              const __grid_constant__ Sums B) {
  __shared__ float sp[WARPS][8];
  __shared__ int sc[WARPS][8];
  __shared__ BlockSum<WARPS> all;
  __shared__ bool last;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = (A.E + 7) / 8;
  const int s = blockIdx.x / blocks, eb = blockIdx.x % blocks, e = eb * 8 + (lane & 7);
  int a = A.offsets ? __ldg(A.offsets + s) : 0, b = A.offsets ? __ldg(A.offsets + s + 1) : A.T;
  if (a < 0 || b < a || b > A.T) {
    if (threadIdx.x == 0) atomicExch(&g_status, kStatusBadOffsets);
    a = min(max(a, 0), A.T);
    b = min(max(b, a), A.T);
  }
  const int64_t first = a / A.per_chunk + s;
  const int chunks = b > a ? (b - 1) / A.per_chunk - a / A.per_chunk + 1 : 0;
  // asked for first, added last: their way from L2 is the same as the others'
  const bool some_here = (int)threadIdx.x < chunks;
  const int n_first = some_here ? A.part_n[first + threadIdx.x] : 0;
  const float z_first = some_here ? A.part_z[first + threadIdx.x] : 0.f;
  float p = 0.f, none = 0.f;
  int c = 0, zero = 0;
#pragma unroll 5
  for (int i = threadIdx.x >> 3; i < chunks; i += WARPS * 4) {
    const int64_t slot = first + i;
    if (e < A.E) {
      p += A.part_p[slot * A.E + e];
      c += A.part_c[slot * A.E + e];
    }
  }
  int n = n_first;
  float z = z_first;
  for (int i = threadIdx.x + WARPS * 32; i < chunks; i += WARPS * 32) {
    n += A.part_n[first + i];
    z += A.part_z[first + i];
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    p += __shfl_xor_sync(0xffffffffu, p, o);
    c += __shfl_xor_sync(0xffffffffu, c, o);
  }
  if (lane < 8) {
    sp[warp][lane] = p;
    sc[warp][lane] = c;
  }
  all.add(z, none, n, zero);
  if (warp == 0) {
    p = 0.f;
    c = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      p += sp[w][lane & 7];
      c += sc[w][lane & 7];
    }
    const float inv = n ? 1.f / (float)n : 0.f;
    p *= inv;
    if (lane < 8 && e < A.E) {
      B.prob[(int64_t)s * A.E + e] = p;
      B.counts[(int64_t)s * A.E + e] = c;
    }
    const float loss = warp_total(lane < 8 && e < A.E ? (float)c * ((float)A.E / (float)A.k) * inv * p : 0.f);
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
  for (int i = threadIdx.x; i < (int)gridDim.x; i += WARPS * 32) loss += __ldcg(B.loss_part + i);
  for (int i = threadIdx.x; i < A.S; i += WARPS * 32) {
    const int m = __ldcg(B.tokens + i);
    z += __ldcg(B.z_part + i);
    n += m;
    some += m > 0;
  }
  all.add(loss, z, n, some);
  if (threadIdx.x == 0) {
    B.losses[0] = some ? loss / (float)some : 0.f;
    B.losses[1] = n ? z / (float)n : 0.f;
    B.totals[0] = some;
    B.totals[1] = n;
  }
}

// The gradient: the same walk over the tokens, a sequence's weights in registers.
template <int N, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kBackThreads) backward_kernel(
    const __grid_constant__ Args A, const float* __restrict__ dlosses,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ totals, int add, float* __restrict__ dlogits) {
  __shared__ Offsets off;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int G = A.group, gl = lane & (G - 1), groups = kBackThreads / G, sub = threadIdx.x / G;
  const int t0 = blockIdx.x * A.per_chunk, t1 = min(A.T, t0 + A.per_chunk);
  Tile<N, VEC> tile;
  tile.ask(A, (int64_t)t0 + sub, t1, gl);
  const int some = __ldg(totals), all = __ldg(totals + 1);
  const float d0 = __ldg(dlosses), d1 = __ldg(dlosses + 1) * 2.f / (float)max(all, 1);
  off.fetch(A);
  float g[N];
  auto weights = [&](int s) {  // of sequence s: d balance / d p
    if (s < 0) return;
    const float n = (float)max(__ldg(tokens + s), 1);
    const float f = d0 * ((float)A.E / (float)A.k) / (n * n * (float)max(some, 1));
    load_lane<N, VEC>((const float*)counts + (int64_t)s * A.E, true, A.E, gl, G, 0.f, g);
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = f * (float)__float_as_int(g[i]);
  };
  int start = t0;
  Run r = off.run(A, t0, t1);
  weights(r.s);
  for (int b = t0; b < t1; b += groups) {
    const int mine = b + sub;
    const bool live = tile.live;
    tile.add_bias(A, gl);
    Token<N, SIGMOID> k;
    k.set(tile.z, G);
    tile.ask(A, (int64_t)mine + groups, t1, gl);
    for (;;) {
      float dot = 0.f;
      if (r.s >= 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) dot = fmaf(g[i], k.p[i], dot);
      }
      dot = group_add(dot, G);
      const bool takes = live && r.s >= 0;
      if (mine >= start && mine < r.end && (takes || !add)) {
        const float dl = d1 * k.lse;
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if constexpr (SIGMOID) v[i] = fmaf(k.p[i] * k.slope[i], g[i] - dot, dl * k.soft[i]);
          else v[i] = k.p[i] * (g[i] - dot + dl);
          if (!takes) v[i] = 0.f;
        }
        float* row = dlogits + (int64_t)mine * A.E;
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            const int e = expert<N, VEC>(i, gl, G);
            if (e >= A.E) break;
            float4 q = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            if (add) {
              const float4 o = *(const float4*)(row + e);
              q.x += o.x; q.y += o.y; q.z += o.z; q.w += o.w;
            }
            *(float4*)(row + e) = q;
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int e = expert<N, VEC>(i, gl, G);
            if (e < A.E) row[e] = add ? row[e] + v[i] : v[i];
          }
        }
      }
      if (r.end >= t1 || r.end - groups > b) break;  // the chunk ends, or the run goes on behind the tile
      start = r.end;
      r = off.run(A, start, t1);
      weights(r.s);
    }
  }
}

// Experts of a lane at most, and lanes of a token.
static int per_lane(int E) { return E <= 4 ? 4 : E <= 8 ? 8 : 16; }
static int group_of(int E) {
  int g = 1;
  while (g * per_lane(E) < E) g <<= 1;
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
  // few tokens: 16 at least, for few partial sums, where a CTA takes as many at once
  A.per_chunk = std::max(std::min(threads / A.group, 16), ceil_div(c.T, ctas));
  return A;
}
static Args forward_args(const moe_balance_t& c, const float* logits) {
  return args_of(c, logits, num_sms() * 2, kThreads);
}
struct Layout {
  size_t p, c, n, z, loss, zs, arrived, total;
};
static Layout layout(const moe_balance_t& c) {
  const Args A = forward_args(c, nullptr);
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
  l.loss = take((size_t)A.S * ceil_div(A.E, 8) * 4);
  l.zs = take((size_t)A.S * 4);
  l.arrived = take(4);
  l.total = at;
  return l;
}

// The kernel instance of a configuration; rows in pieces of four where they are aligned.
#define BALANCE_PICK_N(name, V, S) (c.E <= 4 ? go(name<4, V, S>) : c.E <= 8 ? go(name<8, V, S>) : go(name<16, V, S>))
#define BALANCE_PICK(name, vec)                                                            \
  (A.sigmoid ? (vec ? BALANCE_PICK_N(name, true, true) : BALANCE_PICK_N(name, false, true)) \
             : (vec ? BALANCE_PICK_N(name, true, false) : BALANCE_PICK_N(name, false, false)))
static bool pieces(const Args& A, const void* a, const void* b) {
  return A.E % 4 == 0 && (((uintptr_t)A.logits | (uintptr_t)A.bias | (uintptr_t)a | (uintptr_t)b) & 15) == 0;
}

}  // namespace balance

using namespace balance;

size_t balance_ws_bytes(const moe_balance_t& c) { return layout(c).total; }

moe_status_t launch_balance(const moe_balance_t& c, const float* logits, const int32_t* ids,
                            float* losses, int32_t* counts, int32_t* tokens, float* prob,
                            int32_t* totals, void* ws, cudaStream_t s) {
  Args A = forward_args(c, logits);
  const Layout l = layout(c);
  uint8_t* w = (uint8_t*)ws;
  A.ids = ids;
  A.part_p = (float*)(w + l.p);
  A.part_c = (int32_t*)(w + l.c);
  A.part_n = (int32_t*)(w + l.n);
  A.part_z = (float*)(w + l.z);
  Sums B{losses, prob, counts, tokens, totals, (float*)(w + l.loss), (float*)(w + l.zs), (int*)(w + l.arrived)};
  auto go = [&](auto kern) {
    return launch_k(kern, dim3(ceil_div(c.T, A.per_chunk)), dim3(kThreads), 0, s, (const Args&)A, B.arrived);
  };
  const moe_status_t st = BALANCE_PICK(partial_kernel, pieces(A, nullptr, nullptr));
  if (st != MOE_OK) return st;
  const int blocks = A.S * ceil_div(c.E, 8);
  if (ceil_div(c.T, A.per_chunk) / A.S >= 32)  // slots of a sequence, about
    return launch_k(sequence_kernel<16>, dim3(blocks), dim3(512), 0, s, (const Args&)A, (const Sums&)B);
  return launch_k(sequence_kernel<4>, dim3(blocks), dim3(128), 0, s, (const Args&)A, (const Sums&)B);
}

moe_status_t launch_balance_backward(const moe_balance_t& c, const float* dlosses,
                                     const float* logits, const int32_t* counts,
                                     const int32_t* tokens, const int32_t* totals, int accumulate,
                                     float* dlogits, cudaStream_t s) {
  const Args A = args_of(c, logits, num_sms() * 4, kBackThreads);
  auto go = [&](auto kern) {
    return launch_k(kern, dim3(ceil_div(c.T, A.per_chunk)), dim3(kBackThreads), 0, s, A, dlosses, counts, tokens,
                    totals, accumulate, dlogits);
  };
  return BALANCE_PICK(backward_kernel, pieces(A, counts, dlogits));
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
