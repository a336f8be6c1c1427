// row_ring.cuh — what the norms' kernels (block_norm.cu, layer_norm.cu) share (internal header): rows
// in 16-byte pieces as packed fp32 pairs, a thread's ring of asynchronous copies of its next rows, sums
// over a row's threads, column sums over tokens, and the launch that fits a kernel to an SM.
//
// Persistent CTAs take consecutive rows (several at a time where rows are short), a group of threads
// a row. Each thread copies the pieces of its next rows into shared memory asynchronously (cp.async,
// its own pieces alone, so no barrier guards them) while it works on the current row from registers.
#pragma once

#include "tc_ptx.cuh"
#include "train.cuh"

namespace moe {
namespace rows {

using namespace ptx;

constexpr int kMaxIn = 5;         // row tensors a kernel reads
constexpr int kMaxStages = 3;
constexpr int kMaxThreads = 512;  // of a CTA
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
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
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
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2(0.f, 0.f);
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
// thread c % group; a group takes `rows` consecutive rows at once and a CTA `per` groups' (a unit).
struct Shape {
  int T, H, chunks, group, per, units;
  int rows = 1;
  float scale, offset, eps, inv_h;
  int n_in;           // row tensors read
  int stages;
  const void* in[kMaxIn];
};

// Sums of N values over a row's group, in every thread of it. Every thread of the CTA calls it,
// whether its row exists or not. Two buffers used in turn make one barrier a reduction enough.
struct Reducer {
  float buf[2][4][kMaxThreads / 32];
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
// too long for the ring (kRinged) are read from global memory as they are used. FLAT: rows behind the last
// are zeros, and a thread reads something of a chunk that it does not hold (see get), so that a row's arithmetic
// takes no branches.
template <typename T, int VPT>
constexpr bool kRinged = VPT * (int)sizeof(T) <= 8;

template <typename T, int VPT, int MAXIN, int ROWS = 1, bool FLAT = false>
struct Ring {
  static constexpr bool on = kRinged<T, VPT>;
  const Shape& S;
  const uint8_t* base;
  const uint8_t* mine;    // this thread's first chunk in the current stage
  uint32_t first;         // and in stage 0, as a shared address
  uint32_t tensor_bytes, stage_bytes, step;  // step: from a thread's chunk to its next
  uint32_t row_bytes, off;                   // off: its first chunk inside a row
  bool has[VPT];
  int local, stage = 0;
  __device__ __forceinline__ Ring(const Shape& S_, uint8_t* smem, int local_, int g)
      : S(S_), base(smem), local(local_) {
    static_assert(on || !FLAT, "zeros come through the ring");
    row_bytes = (uint32_t)S.H * sizeof(T);
    tensor_bytes = row_bytes * S.per * ROWS;
    stage_bytes = tensor_bytes * S.n_in;
    step = S.group * Chunk<T>::kBytes;
    off = g * Chunk<T>::kBytes;
    mine = smem + local * ROWS * row_bytes + off;
    first = su32(mine);
#pragma unroll
    for (int v = 0; v < VPT; ++v) has[v] = g + v * S.group < S.chunks;
  }
  __device__ __forceinline__ void issue(int u, int s) {  // one group of copies: unit u into stage s
    if constexpr (on) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        int t = (u * S.per + local) * ROWS + r;
        if (u >= S.units || (!FLAT && t >= S.T)) break;
        uint32_t bytes = 16;
        if (FLAT && t >= S.T) {
          t = 0;
          bytes = 0;
        }
        const int64_t from = (int64_t)t * row_bytes + off;
        uint32_t dst = first + s * stage_bytes + r * row_bytes;
#pragma unroll
        for (int i = 0; i < MAXIN; ++i) {
          if (i >= S.n_in) break;
          const uint8_t* src = (const uint8_t*)S.in[i] + from;
#pragma unroll
          for (int v = 0; v < VPT; ++v) {
            if (has[v]) {
#pragma unroll
              for (int b = 0; b < Chunk<T>::kBytes; b += 16)
                cp_async16(dst + v * step + b, src + v * step + b, bytes);
            }
          }
          dst += tensor_bytes;
        }
      }
      cp_async_commit();
    }
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
  // chunk v of tensor i in row r of the group's rows in the current unit; t: that row. ZEROS: where the thread does
  // not hold the chunk, zeros, otherwise its first chunk of the row, whose values the row's mean and
  // deviation fit: (0 - mean) * rstd can be infinite where no element's value is.
  template <bool ZEROS = true>
  __device__ __forceinline__ void get(Chunk<T>& q, int i, int v, int t, int r = 0) const {
    if (FLAT && v == VPT - 1) {  // only a row's last round of chunks has threads without one
      const uint8_t* row = mine + i * tensor_bytes + r * row_bytes;
      q.load_shared(has[v] ? row + v * step : ZEROS ? base : row);
      if (ZEROS && !has[v]) q.zero();
      return;
    }
    if (on) q.load_shared(mine + i * tensor_bytes + r * row_bytes + v * step);
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

// Where the column sums of `kinds` kinds go: the results themselves when there is one CTA.
struct Outs {
  float* p[3];
};

// A thread's column sums after its last row: the CTA's groups' sums are added in order through shared
// memory (the ring, whose copies have all landed), then leave as a partial row, or as the result of a
// lone CTA. Called by all threads.
template <int VPT>
__device__ __forceinline__ void leave_columns(const Shape& S, uint8_t* smem, int local, int g,
                                              const F2 (&s)[VPT][4], int kind, int kinds,
                                              float factor, float* ws, const Outs& outs) {
  float* to = gridDim.x == 1 ? outs.p[kind] : ws + ((int64_t)blockIdx.x * kinds + kind) * S.H;
  float* all = S.per > 1 ? (float*)smem + (int64_t)local * S.H : to;
  const bool pieces = ((uintptr_t)all & 15) == 0;  // a result need not start on 16 bytes
  if (S.per > 1) __syncthreads();
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = g + v * S.group;
    if (c >= S.chunks) continue;
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      split(s[v][i], f[2 * i], f[2 * i + 1]);
      f[2 * i] *= factor;
      f[2 * i + 1] *= factor;
    }
    if (pieces) {
      float4* at = (float4*)(all + c * 8);
      at[0] = make_float4(f[0], f[1], f[2], f[3]);
      at[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) all[c * 8 + i] = f[i];
    }
  }
  if (S.per == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < S.H; c += blockDim.x) {
    float sum = 0.f;
    for (int l = 0; l < S.per; ++l) sum += ((const float*)smem)[l * S.H + c];
    to[c] = sum;
  }
}

// Column sums of the partial rows: part[rows][kinds][H] -> out[kind][H]. A block takes 32 columns in pieces
// of four: eight threads a row, 32 rows at once; thread group w adds rows w, w + 32, ..., then the 32 sums
// of a column are added in a fixed tree. Small blocks: the rows' way from L2 bounds it.
static __global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ part, int rows,
                                                                int kinds, int H, const Outs out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float4 sh[32][9];
  const int64_t width = (int64_t)kinds * H;
  const int64_t col = (int64_t)blockIdx.x * 32 + (threadIdx.x & 7) * 4;
  float4 s = make_float4(0, 0, 0, 0);
  if (col < width) {
#pragma unroll 8
    for (int r = threadIdx.x >> 3; r < rows; r += 32) {
      const float4 v = *(const float4*)(part + r * width + col);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  sh[threadIdx.x >> 3][threadIdx.x & 7] = s;
  __syncthreads();
  // eight threads a column, 4 sums each: pairs 16 apart, then 8, 4, 2 and 1
  const int c = threadIdx.x >> 3, q = threadIdx.x & 7;
  const float* mine = (const float*)&sh[q][0] + c;
  constexpr int STEP = 8 * 9 * 4;
  float sum = (mine[0] + mine[2 * STEP]) + (mine[STEP] + mine[3 * STEP]);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int64_t to = (int64_t)blockIdx.x * 32 + c;
  if (q == 0 && to < width) out.p[to / H][to % H] = sum;
}
inline moe_status_t launch_column_sum(const float* part, int rows, int kinds, int H, const Outs& outs,
                                      cudaStream_t s) {
  return launch_k(column_sum_kernel, dim3((unsigned)ceil_div64((int64_t)kinds * H, 32)), dim3(256), 0, s, part,
                  rows, kinds, H, outs);
}

// Partial rows at most: the backward kernels' CTAs.
constexpr int kMaxCtas = 4;  // an SM
inline int max_blocks(const Shape& s) { return std::min(s.units, num_sms() * kMaxCtas); }

// Fills in the ring's stages, as many as the budget of an SM's resident CTAs allows. Returns the
// CTA's dynamic shared memory.
inline size_t plan_ring(Shape& s, size_t es, int ctas, bool ringed, size_t budget) {
  const size_t stage = (size_t)s.per * s.rows * s.H * es * s.n_in;
  s.stages = 1;
  if (!ringed) return 0;
  s.stages = (int)std::min<size_t>(kMaxStages, std::max<size_t>(1, budget / ctas / stage));
  return stage * s.stages;
}

template <typename... KArgs, typename... Args>
inline moe_status_t run_within(size_t budget, void (*kern)(KArgs...), Shape& S, size_t es,
                               size_t least, bool ringed, int max_ctas, int& blocks, cudaStream_t s,
                               Args&&... args) {
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
  size_t smem = std::max(plan_ring(S, es, ctas, ringed, budget), least);
  ctas = std::max(1, std::min<int>(ctas, (int)(220 * 1024 / (smem + 1024))));
  blocks = std::min(S.units, num_sms() * ctas);
  return launch_k(kern, dim3(blocks), dim3(threads), smem, s, (const Shape&)S,
                  std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
inline moe_status_t run(void (*kern)(KArgs...), Shape& S, size_t es, size_t least, bool ringed,
                        int max_ctas, int& blocks, cudaStream_t s, Args&&... args) {
  return run_within(kRingBudget, kern, S, es, least, ringed, max_ctas, blocks, s,
                    std::forward<Args>(args)...);
}

}  // namespace rows
}  // namespace moe
