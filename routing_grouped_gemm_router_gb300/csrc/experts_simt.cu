// experts_simt.cu — the experts' products and weight gradients on CUDA cores: fp32 operands
// (tensor-core tf32 keeps 10 bits of them) and the plainest form of the bf16 ones.
//
// One CTA computes a 64 x 64 tile of one expert's product; 256 threads hold 4 x 4 sums each.
// Operand tiles go through shared memory as fp32, 16 of the reduction at a time.
#include "train.cuh"

namespace moe {
namespace esimt {

constexpr int TM = 64, TN = 64, TK = 16, kThreads = 256;

__device__ int g_status;

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }

// The row tile blockIdx.x of the experts' rows: tiles of TM rows, expert by expert; the tiles
// after the last one cover the rows past the experts' runs (e = -1), which are zeroed.
struct Tile {
  int e, row, rows, pad;  // rows that hold slots; pad: rows up to the run's padded end
};
__device__ __forceinline__ Tile find_tile(const int* start, const int* cnt, int E, int rows) {
  int left = blockIdx.x;
  for (int e = 0; e < E; ++e) {
    const int n = (cnt[e] + TM - 1) / TM;
    if (left < n) {
      const int r = cnt[e] - left * TM;
      const int end = min(start[e] + (cnt[e] + kRowBlock - 1) / kRowBlock * kRowBlock, rows);
      return {e, start[e] + left * TM, min(r, TM), min(end - (start[e] + left * TM), TM)};
    }
    left -= n;
  }
  const int row = start[E] + min(left, (rows - start[E]) / TM + 1) * TM;
  return {-1, row, 0, max(0, min(rows - row, TM))};
}

// C[rows, N] = A[rows, K] * W[e], W[e] given as [N, K] (TRANS = false: products with W^T) or
// [K, N] (TRANS). KIND up keeps two sums (rows n and N + n of W13) and writes h13 and act.
template <typename T, int KIND>
__global__ void __launch_bounds__(kThreads) product_kernel(
    const T* __restrict__ A, const T* __restrict__ W, const float* __restrict__ h13,
    const int32_t* __restrict__ counts, int E, int rows, int N, int K, void* __restrict__ out_,
    T* __restrict__ act) {
  pdl_wait();
  pdl_trigger();
  constexpr bool TRANS = KIND == kDownGrad || KIND == kUpGrad;
  constexpr int D = KIND == kUp ? 2 : 1;  // sums a thread keeps per element
  T* out = (T*)out_;
  __shared__ int start[kMaxExperts + 1], cnt[kMaxExperts];
  __shared__ float sA[TK][TM + 4], sB[D][TK][TN + 4];
  load_counts(counts, E, cnt);
  __syncthreads();
  if (threadIdx.x < 32) expert_rows(E, rows, start, cnt, &g_status);
  __syncthreads();
  const Tile tl = find_tile(start, cnt, E, rows);
  if (tl.pad <= 0) return;
  const int n0 = blockIdx.y * TN;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[D][4][4] = {};
  if (tl.e >= 0) {
    const T* We = W + (int64_t)tl.e * D * N * K;
    for (int k0 = 0; k0 < K; k0 += TK) {
      for (int i = threadIdx.x; i < TM * TK; i += kThreads) {
        const int m = i / TK, kk = i % TK;
        sA[kk][m] = m < tl.rows && k0 + kk < K ? to_f(A[(int64_t)(tl.row + m) * K + k0 + kk]) : 0.f;
      }
#pragma unroll
      for (int d = 0; d < D; ++d)
        for (int i = threadIdx.x; i < TN * TK; i += kThreads) {
          const int n = TRANS ? i % TN : i / TK, kk = TRANS ? i / TN : i % TK;
          float v = 0.f;
          if (n0 + n < N && k0 + kk < K)
            v = to_f(TRANS ? We[(int64_t)(k0 + kk) * N + n0 + n]
                           : We[((int64_t)d * N + n0 + n) * K + k0 + kk]);
          sB[d][kk][n] = v;
        }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < TK; ++kk) {
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = sA[kk][ty * 4 + i];
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float b = sB[d][kk][tx * 4 + j];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[d][i][j] = fmaf(a[i], b, acc[d][i][j]);
          }
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = ty * 4 + i;
    if (m >= tl.pad) continue;
    const bool slot = m < tl.rows;
    const int64_t p = tl.row + m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= N) continue;
      const float v = slot ? acc[0][i][j] : 0.f;
      if (KIND == kUp) {
        const float u = slot ? acc[D - 1][i][j] : 0.f;
        ((float*)out_)[p * 2 * N + n] = v;
        ((float*)out_)[p * 2 * N + N + n] = u;
        act[p * N + n] = from_f<T>(v * sigmoid(v) * u);
      } else if (KIND == kDownGrad) {
        const float g = slot ? h13[p * 2 * N + n] : 0.f;
        const float u = slot ? h13[p * 2 * N + N + n] : 0.f;
        const float s = sigmoid(g);
        out[p * 2 * N + n] = from_f<T>(v * u * s * (1.f + g * (1.f - s)));
        out[p * 2 * N + N + n] = from_f<T>(v * g * s);
        act[p * N + n] = from_f<T>(g * s * u);
      } else {
        out[p * N + n] = from_f<T>(v);
      }
    }
  }
}

// dW[e][m, n] (+)= sum over expert e's rows p of dy[p, m] a[p, n].
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) weight_grad_kernel(
    const T* __restrict__ dy, const T* __restrict__ a, const int32_t* __restrict__ counts, int E,
    int rows, int M, int N, int accumulate, O* __restrict__ dW) {
  pdl_wait();
  pdl_trigger();
  __shared__ int start[kMaxExperts + 1], cnt[kMaxExperts];
  __shared__ float sA[TK][TM], sB[TK][TN];
  load_counts(counts, E, cnt);
  __syncthreads();
  if (threadIdx.x < 32) expert_rows(E, rows, start, cnt, &g_status);
  __syncthreads();
  const int tn = (N + TN - 1) / TN, tm = (M + TM - 1) / TM;
  const int e = blockIdx.x / (tn * tm), rest = blockIdx.x % (tn * tm);
  const int m0 = rest / tn * TM, n0 = rest % tn * TN;
  const int p0 = start[e], np = cnt[e];
  if (np == 0 && accumulate) return;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < np; k0 += TK) {
    for (int i = threadIdx.x; i < TK * TM; i += kThreads) {
      const int kk = i / TM, m = i % TM;
      const int64_t p = p0 + k0 + kk;
      sA[kk][m] = k0 + kk < np && m0 + m < M ? to_f(dy[p * M + m0 + m]) : 0.f;
      sB[kk][m] = k0 + kk < np && n0 + m < N ? to_f(a[p * N + n0 + m]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < TK; ++kk) {
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = sA[kk][ty * 4 + i];
        y[i] = sB[kk][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= M || n >= N) continue;
      O* o = dW + ((int64_t)e * M + m) * N + n;
      *o = from_f<O>(accumulate ? to_f(*o) + acc[i][j] : acc[i][j]);
    }
}

}  // namespace esimt

using namespace esimt;

template <typename T>
static moe_status_t product(ExpertProduct kind, const moe_experts_t& c, const void* a,
                            const void* w, const float* h13, const int32_t* counts, void* out,
                            void* act, cudaStream_t s) {
  const int N = kind == kUp || kind == kDownGrad ? c.I : c.H;
  const int K = kind == kUp || kind == kDownGrad ? c.H : kind == kDown ? c.I : 2 * c.I;
  // row tiles: at most one partly filled one an expert, and the rows past the last run
  const dim3 grid(2 * ceil_div(c.rows, TM) + c.E, ceil_div(N, TN));
  auto go = [&](auto kern) {
    return launch_k(kern, grid, dim3(kThreads), 0, s, (const T*)a, (const T*)w,
                    h13, counts, c.E, c.rows, N, K, out, (T*)act);
  };
  switch (kind) {
    case kUp: return go(product_kernel<T, kUp>);
    case kDown: return go(product_kernel<T, kDown>);
    case kDownGrad: return go(product_kernel<T, kDownGrad>);
    default: return go(product_kernel<T, kUpGrad>);
  }
}

moe_status_t launch_expert_product_simt(ExpertProduct kind, const moe_experts_t& c, const void* a,
                                        const void* w, const float* h13, const int32_t* counts,
                                        void* out, void* act, cudaStream_t s) {
  return c.dtype == MOE_BF16 ? product<__nv_bfloat16>(kind, c, a, w, h13, counts, out, act, s)
                             : product<float>(kind, c, a, w, h13, counts, out, act, s);
}

moe_status_t launch_weight_grad_simt(int rows, int E, int M, int N, moe_dtype_t dt,
                                     moe_dtype_t out_dt, int accumulate, const void* dy,
                                     const void* a, const int32_t* counts, void* dW,
                                     cudaStream_t s) {
  const int64_t tiles = (int64_t)E * ceil_div(M, TM) * ceil_div(N, TN);
  if (tiles > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  auto go = [&](auto kern, auto* d, auto* x, auto* o) {
    return launch_k(kern, dim3((unsigned)tiles), dim3(kThreads), 0, s, d, x, counts, E, rows, M, N,
                    accumulate, o);
  };
  using bf = __nv_bfloat16;
  if (dt == MOE_F32)
    return go(weight_grad_kernel<float, float>, (const float*)dy, (const float*)a, (float*)dW);
  if (out_dt == MOE_F32)
    return go(weight_grad_kernel<bf, float>, (const bf*)dy, (const bf*)a, (float*)dW);
  return go(weight_grad_kernel<bf, bf>, (const bf*)dy, (const bf*)a, (bf*)dW);
}

int train_status_read(int reset) {
  int v = 0;
  cudaMemcpyFromSymbol(&v, g_status, sizeof(int));
  if (reset) {
    int z = 0;
    cudaMemcpyToSymbol(g_status, &z, sizeof(int));
  }
  const int t = experts_tc_status_read(reset);
  return t ? t : v;
}

}  // namespace moe
