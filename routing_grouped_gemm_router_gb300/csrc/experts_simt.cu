// experts_simt.cu — the experts' fp32 products and weight gradients on CUDA cores (tensor-core
// tf32 keeps 10 bits of an operand, and a sum of split bf16 products loses the low bits of long
// reductions).
//
// One CTA computes a TM x 128 tile of one expert's product, 256 threads with 8 x 8 sums each (TM =
// 128) or 128 with 4 x 8 (TM = 32). Operand
// tiles of 16 reduction steps are loaded into registers while the previous ones are used (two
// buffers, one barrier a tile). TM is 128 where experts have many rows; with few, 32-row tiles
// keep the wasted multiply-adds below the time the weights take from HBM. The FMA pipes bound it.
//
// A sum of n products in a row is off by about 0.3 sqrt(n) half units of fp32 (2.2e-6 of the result
// measured over 15,600 steps; so 8e-7 over 2048). Reductions of more than kLong steps (LONG) are summed in spans of
// kSpan steps, whose sums are added to totals in shared memory: 4e-7 at any length. The registers are
// full, so a branch in the loop costs more than the additions: 4096 steps 5 to 11 % (up 9480 -> 10,020 us for
// 8 experts of 4096 x 4096 over 1024 rows, down 4850 -> 5360), weight gradients 2 %; shorter ones do without.
#include "train.cuh"

namespace moe {
namespace esimt {

constexpr int TN = 128, TK = 16;
constexpr int PAD = 4;
constexpr int kLong = 2048;  // steps from which on a reduction is summed in spans
constexpr int kSpan = 512;   // steps of a span (a multiple of TK)

__device__ int g_status;

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }

// A tile of ROWS x TK values of a matrix whose reduction index is contiguous (KC) or whose other
// index is: into registers, then into shared memory as s[k][row]. Rows from `limit` on and reduction
// steps from `kmax` on are zeros. Both limits and ld are multiples of 4 along the contiguous index
// (H and I are multiples of 8; the reduction over an expert's rows runs over the other one).
template <int ROWS, bool KC, int THREADS>
struct Tile {
  static constexpr int COUNT = ROWS * TK / 4 / THREADS;  // float4 a thread
  static_assert(COUNT >= 1 && COUNT * THREADS * 4 == ROWS * TK, "whole pieces");
  float4 r[COUNT];
  __device__ __forceinline__ void load(const float* __restrict__ p, int64_t ld, int limit, int k0,
                                       int kmax) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int f = threadIdx.x + i * THREADS;
      r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int row = KC ? f / (TK / 4) : f % (ROWS / 4) * 4;
      const int k = KC ? f % (TK / 4) * 4 : f / (ROWS / 4);
      if (row < limit && k0 + k < kmax)
        r[i] = __ldg((const float4*)(KC ? p + row * ld + k0 + k : p + (k0 + k) * ld + row));
    }
  }
  template <int W>
  __device__ __forceinline__ void store(float (*s)[W], int col0) const {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const int f = threadIdx.x + i * THREADS;
      if (KC) {
        const int row = col0 + f / (TK / 4), k = f % (TK / 4) * 4;
        s[k][row] = r[i].x;
        s[k + 1][row] = r[i].y;
        s[k + 2][row] = r[i].z;
        s[k + 3][row] = r[i].w;
      } else {
        const int row = col0 + f % (ROWS / 4) * 4, k = f / (ROWS / 4);
        *(float4*)&s[k][row] = r[i];
      }
    }
  }
};

// acc[i][j] += sum over a tile's 16 steps of rows ty * MR + 2i, + 1 of a times column j of this
// thread. Its eight columns are tx * 4 .. + 3 and 64 + tx * 4 .. + 3. Pairs of rows share an
// instruction, which leaves issue slots for everything else.
template <int MR, int TM>
__device__ __forceinline__ void multiply(const float (*a)[TM + PAD], const float (*b)[TN + PAD],
                                         F2 (&acc)[MR / 2][8]) {
  static_assert(MR % 4 == 0, "whole pieces of a column");
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int k = 0; k < TK; ++k) {
    F2 x[MR / 2];
    float y[8];
#pragma unroll
    for (int i = 0; i < MR; i += 4) {
      const float4 q = *(const float4*)&a[k][ty * MR + i];
      x[i / 2] = f2(q.x, q.y);
      x[i / 2 + 1] = f2(q.z, q.w);
    }
    *(float4*)&y[0] = *(const float4*)&b[k][tx * 4];
    *(float4*)&y[4] = *(const float4*)&b[k][64 + tx * 4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const F2 yy = f2(y[j], y[j]);
#pragma unroll
      for (int i = 0; i < MR / 2; ++i) acc[i][j] = fma2(x[i], yy, acc[i][j]);
    }
  }
}
// A thread's totals of the spans so far, a float4 every blockDim.x of them.
template <int MR>
struct Totals {
  float4* mine;
  bool any = false;
  __device__ __forceinline__ explicit Totals(float4* smem) : mine(smem + threadIdx.x) {}
  // sums += the totals so far
  __device__ __forceinline__ void add_to(F2 (&sums)[MR / 2][8]) const {
    if (!any) return;
#pragma unroll
    for (int c = 0; c < MR * 2; ++c) {
      const float4 q = mine[c * blockDim.x];
      F2 &a = sums[c / 4][c % 4 * 2], &b = sums[c / 4][c % 4 * 2 + 1];
      a = a + f2(q.x, q.y);
      b = b + f2(q.z, q.w);
    }
  }
  // the totals take the sums in, which start again
  __device__ __forceinline__ void take(F2 (&sums)[MR / 2][8]) {
    add_to(sums);
#pragma unroll
    for (int c = 0; c < MR * 2; ++c) {
      F2 &a = sums[c / 4][c % 4 * 2], &b = sums[c / 4][c % 4 * 2 + 1];
      float4 q;
      split(a, q.x, q.y);
      split(b, q.z, q.w);
      mine[c * blockDim.x] = q;
      a = b = f2(0.f, 0.f);
    }
    any = true;
  }
};
template <int MR>
__device__ __forceinline__ void unpair(const F2 (&p)[MR / 2][8], float (&acc)[MR][8]) {
#pragma unroll
  for (int i = 0; i < MR / 2; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) split(p[i][j], acc[2 * i][j], acc[2 * i + 1][j]);
}

struct Rows {
  int e, row, rows, pad;  // expert; first row; rows that hold slots; rows up to the padded end
};

// C[rows, N] = A[rows, K] * W[e], W[e] given as [N, K] (up, down) or [K, N] (their gradients).
// The columns of an up tile are 64 gate rows of W13 and the same 64 up rows. Row tiles after the last
// expert's cover the rows past the experts' runs, which are zeroed.
template <int TM>
constexpr int kThreadsOf = TM == 128 ? 256 : 128;

template <int KIND, int TM, bool LONG>
__global__ void __launch_bounds__(kThreadsOf<TM>, TM == 128 ? 2 : 4) product_kernel(
    const float* __restrict__ A, const float* __restrict__ W, const float* __restrict__ h13,
    const int32_t* __restrict__ counts, int E, int rows, int N, int K, float* __restrict__ out,
    float* __restrict__ act) {
  pdl_wait();
  pdl_trigger();
  constexpr bool TRANS = KIND == kDownGrad || KIND == kUpGrad;
  constexpr int kThreads = kThreadsOf<TM>;
  constexpr int MR = TM / (kThreads / 16);
  constexpr int CN = KIND == kUp ? 64 : 128;  // output columns of a tile
  extern __shared__ __align__(16) float4 smem_totals[];  // LONG
  __shared__ int start[kMaxExperts + 1], cnt[kMaxExperts];
  __shared__ Rows tile;
  __shared__ __align__(16) float sA[2][TK][TM + PAD], sB[2][TK][TN + PAD];
  load_counts(counts, E, cnt);
  __syncthreads();
  if (threadIdx.x < 32) {
    expert_rows(E, rows, start, cnt, &g_status);
    __syncwarp();
    // the expert whose tile this is: tiles of lower experts are counted 32 experts at a time
    const int lane = threadIdx.x, want = blockIdx.x;
    int before = 0;
    bool found = false;
    for (int e0 = 0; e0 < E && !found; e0 += 32) {
      const int e = e0 + lane, n = e < E ? (cnt[e] + TM - 1) / TM : 0;
      int inc = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
      }
      const int lo = before + inc - n;
      const bool here = want >= lo && want < lo + n;
      if (here) {
        const int at = (want - lo) * TM;
        const int end = min((cnt[e] + kRowBlock - 1) / kRowBlock * kRowBlock, rows - start[e]);
        tile = {e, start[e] + at, min(cnt[e] - at, TM), min(end - at, TM)};
      }
      found = __any_sync(0xffffffffu, here);
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (!found && lane == 0) {
      const int64_t row = start[E] + (int64_t)(want - before) * TM;
      tile = {-1, (int)min(row, (int64_t)rows), 0, (int)max((int64_t)0, min(rows - row, (int64_t)TM))};
    }
  }
  __syncthreads();
  const Rows tl = tile;
  if (tl.pad <= 0) return;
  const int n0 = blockIdx.y * CN;
  F2 sums[MR / 2][8] = {};
  if (tl.e >= 0) {
    Totals<MR> totals(smem_totals);
    const float* We = W + (int64_t)tl.e * (KIND == kUp ? 2 : 1) * N * K;
    const float* Ar = A + (int64_t)tl.row * K;
    Tile<TM, true, kThreads> ta;
    // two half tiles of columns: gate and up rows, or 128 columns in a row
    Tile<64, !TRANS, kThreads> tb[2];
    const float* b0 = TRANS ? We + n0 : We + (int64_t)n0 * K;
    const float* b1 = TRANS ? b0 + 64 : KIND == kUp ? b0 + (int64_t)N * K : b0 + (int64_t)64 * K;
    const int64_t ldb = TRANS ? N : K;
    const int lim0 = N - n0, lim1 = KIND == kUp ? N - n0 : N - n0 - 64;
    auto load = [&](int k0) {
      ta.load(Ar, K, tl.rows, k0, K);
      tb[0].load(b0, ldb, lim0, k0, K);
      tb[1].load(b1, ldb, lim1, k0, K);
    };
    auto store = [&](int s) {
      ta.store(sA[s], 0);
      tb[0].store(sB[s], 0);
      tb[1].store(sB[s], 64);
    };
    load(0);
    store(0);
    __syncthreads();
    int s = 0;
    for (int k0 = 0; k0 < K; k0 += TK) {
      const bool more = k0 + TK < K;
      if (more) load(k0 + TK);
      multiply<MR, TM>(sA[s], sB[s], sums);
      if (more) store(s ^ 1);
      if (LONG && more && (k0 + TK) % kSpan == 0) totals.take(sums);
      __syncthreads();
      s ^= 1;
    }
    if (LONG) totals.add_to(sums);
  }
  float acc[MR][8];
  unpair<MR>(sums, acc);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < MR; ++i) {
    const int m = ty * MR + i;
    if (m >= tl.pad) continue;
    const bool slot = m < tl.rows;
    const int64_t p = tl.row + m;
    if (!slot) {
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    }
    if (KIND == kUp) {
      const int n = n0 + tx * 4;
      if (n >= N) continue;
      float a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = acc[i][j] * sigmoid(acc[i][j]) * acc[i][4 + j];
      *(float4*)(out + p * 2 * N + n) = *(const float4*)&acc[i][0];
      *(float4*)(out + p * 2 * N + N + n) = *(const float4*)&acc[i][4];
      *(float4*)(act + p * N + n) = *(const float4*)a;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = n0 + h * 64 + tx * 4;
        if (n >= N) continue;
        if (KIND == kDownGrad) {
          float g[4] = {}, u[4] = {}, a[4];
          if (slot) {
            *(float4*)g = __ldg((const float4*)(h13 + p * 2 * N + n));
            *(float4*)u = __ldg((const float4*)(h13 + p * 2 * N + N + n));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float d = acc[i][4 * h + j], s = sigmoid(g[j]);
            a[j] = g[j] * s * u[j];
            u[j] = d * u[j] * s * (1.f + g[j] * (1.f - s));
            g[j] = d * g[j] * s;
          }
          *(float4*)(out + p * 2 * N + n) = *(const float4*)u;
          *(float4*)(out + p * 2 * N + N + n) = *(const float4*)g;
          *(float4*)(act + p * N + n) = *(const float4*)a;
        } else {
          *(float4*)(out + p * N + n) = *(const float4*)&acc[i][4 * h];
        }
      }
    }
  }
}

// dW[e][m, n] (+)= sum over expert e's rows p of dy[p, m] a[p, n].
template <bool LONG>
__global__ void __launch_bounds__(256, 2) weight_grad_kernel(
    const float* __restrict__ dy, const float* __restrict__ a, const int32_t* __restrict__ counts,
    int E, int rows, int M, int N, int accumulate, float* __restrict__ dW) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) float4 smem_totals[];  // LONG
  __shared__ int start[kMaxExperts + 1], cnt[kMaxExperts];
  __shared__ __align__(16) float sA[2][TK][TN + PAD], sB[2][TK][TN + PAD];
  load_counts(counts, E, cnt);
  __syncthreads();
  if (threadIdx.x < 32) expert_rows(E, rows, start, cnt, &g_status);
  __syncthreads();
  const int tn = (N + TN - 1) / TN, tm = (M + TN - 1) / TN;
  const int e = blockIdx.x / (tn * tm), rest = blockIdx.x % (tn * tm);
  const int m0 = rest / tn * TN, n0 = rest % tn * TN;
  const int np = cnt[e];
  if (np == 0 && accumulate) return;
  F2 sums[4][8] = {};
  if (np > 0) {
    Totals<8> totals(smem_totals);
    const float* dp = dy + (int64_t)start[e] * M + m0;
    const float* ap = a + (int64_t)start[e] * N + n0;
    Tile<TN, false, 256> ta, tb;
    ta.load(dp, M, M - m0, 0, np);
    tb.load(ap, N, N - n0, 0, np);
    ta.store(sA[0], 0);
    tb.store(sB[0], 0);
    __syncthreads();
    int s = 0;
    for (int k0 = 0; k0 < np; k0 += TK) {
      const bool more = k0 + TK < np;
      if (more) {
        ta.load(dp, M, M - m0, k0 + TK, np);
        tb.load(ap, N, N - n0, k0 + TK, np);
      }
      multiply<8, TN>(sA[s], sB[s], sums);
      if (more) {
        ta.store(sA[s ^ 1], 0);
        tb.store(sB[s ^ 1], 0);
      }
      if (LONG && more && (k0 + TK) % kSpan == 0) totals.take(sums);
      __syncthreads();
      s ^= 1;
    }
    if (LONG) totals.add_to(sums);
  }
  float acc[8][8];
  unpair<8>(sums, acc);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + ty * 8 + i;
    if (m >= M) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + h * 64 + tx * 4;
      if (n >= N) continue;
      float4* o = (float4*)(dW + ((int64_t)e * M + m) * N + n);
      float4 v = *(const float4*)&acc[i][4 * h];
      if (accumulate) {
        const float4 w = *o;
        v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
      }
      *o = v;
    }
  }
}

// Leave to use that much dynamic shared memory for the totals.
template <typename K>
static bool totals_fit(K kern, size_t bytes) {
  return bytes == 0 || cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
                           cudaSuccess;
}

}  // namespace esimt

using namespace esimt;

// 32-row tiles below this many buffer rows an expert, 128-row tiles from it on. Measured with 64
// experts of H = 2048, I = 1408, forward and backward: 31 rows an expert 2.70 against 5.98 ms, 79 rows
// 5.91 and 6.92, 143 rows 10.35 and 10.27; 8 experts of 1038 rows 9.42 and 8.22 (51.7 TFLOP/s, 0.93 of
// a batched library product over the same rows).
constexpr int kManyRows = 128;

moe_status_t launch_expert_product_simt(ExpertProduct kind, const moe_experts_t& c, const void* a,
                                        const void* w, const float* h13, const int32_t* counts,
                                        void* out, void* act, cudaStream_t s) {
  const int N = kind == kUp || kind == kDownGrad ? c.I : c.H;
  const int K = kind == kUp || kind == kDownGrad ? c.H : kind == kDown ? c.I : 2 * c.I;
  const bool many = c.rows / c.E >= kManyRows;
  const int tm = many ? 128 : 32;
  // row tiles: full ones, at most one partly filled one an expert, and as many again for the rows past
  // the last run
  const dim3 grid(2 * ceil_div(c.rows, tm) + c.E, ceil_div(N, kind == kUp ? 64 : 128));
  if (grid.y > 65535) return MOE_ERR_UNSUPPORTED;
  const bool lng = K > kLong;
  const int threads = many ? 256 : 128;
  const size_t smem = lng ? (size_t)tm * TN * sizeof(float) : 0;
  auto go = [&](auto kern) {
    if (!totals_fit(kern, smem)) return MOE_ERR_CUDA;
    return launch_k(kern, grid, dim3(threads), smem, s, (const float*)a, (const float*)w, h13, counts, c.E,
                    c.rows, N, K, (float*)out, (float*)act);
  };
#define ESIMT_PICK(kind)                                                                          \
  (many ? (lng ? go(product_kernel<kind, 128, true>) : go(product_kernel<kind, 128, false>))      \
        : (lng ? go(product_kernel<kind, 32, true>) : go(product_kernel<kind, 32, false>)))
  switch (kind) {
    case kUp: return ESIMT_PICK(kUp);
    case kDown: return ESIMT_PICK(kDown);
    case kDownGrad: return ESIMT_PICK(kDownGrad);
    default: return ESIMT_PICK(kUpGrad);
  }
#undef ESIMT_PICK
}

moe_status_t launch_weight_grad_simt(int rows, int E, int M, int N, int accumulate,
                                     const void* dy, const void* a, const int32_t* counts,
                                     void* dW, cudaStream_t s) {
  const int64_t tiles = (int64_t)E * ceil_div(M, TN) * ceil_div(N, TN);
  if (tiles > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  const size_t smem = rows > kLong ? (size_t)TN * TN * sizeof(float) : 0;
  auto go = [&](auto kern) {
    if (!totals_fit(kern, smem)) return MOE_ERR_CUDA;
    return launch_k(kern, dim3((unsigned)tiles), dim3(256), smem, s, (const float*)dy, (const float*)a, counts,
                    E, rows, M, N, accumulate, (float*)dW);
  };
  return smem ? go(weight_grad_kernel<true>) : go(weight_grad_kernel<false>);
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
