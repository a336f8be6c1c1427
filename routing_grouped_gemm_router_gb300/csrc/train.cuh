// train.cuh — shared helpers of the training operators (internal header): 16-byte pieces as
// fp32 values, warp and group sums, the experts' row layout, launch declarations.
#pragma once

#include "common.cuh"
#include "moe_train.h"

namespace moe {

enum : int { kStatusBadCounts = 4 };  // counts that do not fit in the row buffers

// ------------------------------------------------------------------- 16-byte pieces
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static __device__ __forceinline__ void unpack(const uint4& q, float (&f)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint4 q;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return q;
  }
};
template <>
struct Vec<float> {
  static __device__ __forceinline__ void unpack(const uint4& q, float (&f)[4]) {
    f[0] = __uint_as_float(q.x);
    f[1] = __uint_as_float(q.y);
    f[2] = __uint_as_float(q.z);
    f[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// ------------------------------------------------------------------- packed fp32
// Two fp32 values that one instruction works on.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// ------------------------------------------------------------------- experts' rows
constexpr int kRowBlock = MOE_TRAIN_BLOCK;
constexpr int kMaxExperts = 512;
constexpr int kMaxRows = 1 << 28;  // rows of a buffer: the sums below stay in 32 bits

// Counts into shared memory by the whole block; the caller synchronises before expert_rows.
__device__ __forceinline__ void load_counts(const int32_t* __restrict__ counts, int E, int* cnt) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = __ldg(counts + e);
}

// Where expert e's rows start and how many there are, for all experts, in shared memory:
// start[e] = sum over lower experts of their counts (in cnt) rounded up to kRowBlock, both cut to
// fit in `rows` rows. start[E] is the end of the last run. Called by one whole warp; the caller
// synchronises.
__device__ __forceinline__ void expert_rows(int E, int rows, int* start, int* cnt, int* status) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  bool bad = false;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    int c = e < E ? cnt[e] : 0;
    if (c < 0 || c > rows) {
      bad = true;
      c = c < 0 ? 0 : rows;
    }
    const int pad = (c + kRowBlock - 1) / kRowBlock * kRowBlock;
    int inc = pad;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc = min(inc + o, (1 << 30) - 1);
    }
    const int s = min(base + inc - pad, rows);
    if (s + c > rows) {
      bad = true;
      c = rows - s;
    }
    if (e < E) {
      start[e] = s;
      cnt[e] = c;
    }
    base = min(base + __shfl_sync(0xffffffffu, inc, 31), rows);
  }
  if (lane == 0) start[E] = base;
  if (bad && status) atomicExch(status, kStatusBadCounts);
}

// ------------------------------------------------------------------- launches
moe_status_t launch_permute(const void* x, const int32_t* ids, const int32_t* sid, int T, int k,
                            int E, int H, moe_dtype_t dt, int rows, void* xs, int32_t* pos,
                            cudaStream_t s);
moe_status_t launch_slot_sum(const void* ys, const int32_t* pos, const float* w, int T, int k,
                             int H, moe_dtype_t dt, int rows, void* out, cudaStream_t s);
moe_status_t launch_unpermute_backward(const void* dout, const void* ys, const int32_t* sid,
                                       const int32_t* pos, const float* w, int T, int k, int H,
                                       moe_dtype_t dt, int rows, void* dys, float* dw,
                                       cudaStream_t s);

// Products of the experts' rows; which one is kind. up: xs W13^T with the SwiGLU; down:
// act W2^T; down_grad: dys W2 with the SwiGLU's gradient; up_grad: dh13 W13.
enum ExpertProduct { kUp = 0, kDown = 1, kDownGrad = 2, kUpGrad = 3 };
moe_status_t launch_expert_product_simt(ExpertProduct kind, const moe_experts_t& c, const void* a,
                                        const void* w, const float* h13, const int32_t* counts,
                                        void* out, void* act, cudaStream_t s);
moe_status_t launch_expert_product_tc(ExpertProduct kind, const moe_experts_t& c, const void* a,
                                      const void* w, const float* h13, const int32_t* counts,
                                      void* out, void* act, cudaStream_t s);
moe_status_t launch_weight_grad_tc(int rows, int E, int M, int N, moe_dtype_t out_dt,
                                   int accumulate, const void* dy, const void* a,
                                   const int32_t* counts, void* dW, cudaStream_t s);
int experts_tc_status_read(int reset);
moe_status_t launch_weight_grad_simt(int rows, int E, int M, int N, int accumulate,
                                     const void* dy, const void* a, const int32_t* counts,
                                     void* dW, cudaStream_t s);

struct BlockNormArgs {  // pointers of the forward and backward norm and join kernels
  const void *x, *y, *gate, *dres, *dh, *out_in;
  const float *gamma, *gamma_next, *rstd_y_in, *rstd_out_in;
  void *out, *h, *dx, *dy, *dgate;
  float *rstd_y, *rstd_out, *dgamma, *dgamma_next;
  float* ws;
};
size_t block_norm_ws_bytes(const moe_block_t& c);
moe_status_t launch_block_norm(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s);
moe_status_t launch_block_join(const moe_block_t& c, const BlockNormArgs& a, cudaStream_t s);
moe_status_t launch_block_norm_backward(const moe_block_t& c, const BlockNormArgs& a,
                                        cudaStream_t s);
moe_status_t launch_block_join_backward(const moe_block_t& c, const BlockNormArgs& a,
                                        cudaStream_t s);
moe_status_t launch_route_backward(const moe_config_t& c, const float* logits,
                                   const int32_t* ids, const float* dw, float* dlogits,
                                   cudaStream_t s);

int train_status_read(int reset);

}  // namespace moe
