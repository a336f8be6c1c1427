// embed.cu — the embedding lookup and its gradient (moe_embed, moe_embed_backward).
//
//   out[t] = scale table[tok[t]]          dtable[v] (+)= scale sum_{t: tok[t] = v} dx[t]
//
// Both move rows and do next to no arithmetic: HBM bounds them. The gradient's sum has to be the same
// every run, and a token's rows lie anywhere, so the tokens are sorted first (stably, by id) and runs
// of one id summed in that order, in fp32:
//   sort_fill  one CTA, or a cluster of 8, sorts (id, t) by radix passes of up to 9 bits; the other CTAs
//              write the zeros of ids that do not occur meanwhile, most of what a dense gradient writes
//   run_sum    a warp sums 16 sorted rows in a slice of 32 pieces of 16 bytes, and writes every run that
//              lies inside; a run that crosses to other warps' rows leaves fp32 partial sums
//   join       the partial sums of a run are added in order: a run of any length is spread over as many
//              warps as it has rows / 16
// 8192 tokens into 32000 x 4096 in fp32 (591 MB) 75 us of zeros, 26 of sums, 7 of joins; added to a gradient
// that is there, 44 (174 MB) with 9 of sorting.
#include "stack.cuh"
#include "tc_ptx.cuh"
#include "train.cuh"

namespace moe {
namespace embedding {

using namespace ptx;

template <bool WIDE>
__device__ __forceinline__ int id_of(const void* tokens, int64_t t, int V) {  // V: no id
  if (WIDE) {
    const long long v = __ldg((const long long*)tokens + t);
    return v >= 0 && v < V ? (int)v : V;
  }
  const int v = __ldg((const int*)tokens + t);
  return v >= 0 && v < V ? v : V;
}

// ------------------------------------------------------------------- lookup
// A warp takes P pieces a lane of a token's row at a time. Few tokens: one piece a lane, to spread
// over more warps. 16384 tokens of 7168 channels in bf16 52 us: 94 MB of rows read, 235 MB written, 6.3 TB/s.
template <typename T, bool WIDE, int P>
__global__ void __launch_bounds__(256) embed_kernel(const void* __restrict__ tokens, int n,
                                                    const uint4* __restrict__ table, int V, int vec,
                                                    float scale, uint4* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  constexpr int W = 16 / sizeof(T);
  const int v0 = blockIdx.y * (32 * P) + (threadIdx.x & 31);
  for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < n; t += (int64_t)gridDim.x * 8) {
    const int id = id_of<WIDE>(tokens, t, V);
    uint4 q[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      q[p] = make_uint4(0, 0, 0, 0);
      if (id < V && v0 + p * 32 < vec) q[p] = __ldg(table + (int64_t)id * vec + v0 + p * 32);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (v0 + p * 32 >= vec) break;
      float f[W];
      Vec<T>::unpack(q[p], f);
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = id < V ? f[i] * scale : 0.f;
      __stcs(out + t * vec + v0 + p * 32, Vec<T>::pack(f));
    }
  }
}

// ------------------------------------------------------------------- sorting, and zeros
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kHeld = 8;         // keys that a thread holds in registers
constexpr int kHeldCta = kSortThreads * kHeld;
constexpr int kCluster = 8;      // CTAs that sort together
constexpr int kAloneUpTo = 2048; // tokens that one CTA sorts by itself
constexpr int kDigit = 9;        // bits of a pass at most
constexpr int kBins = 1 << kDigit;
constexpr int kFillRows = 1 << 16;   // rows whose marks fit the fill CTAs' shared memory
constexpr int kZeroBytes = 1 << 14;  // zeros that one bulk copy writes at most

struct SortArgs {
  const void* tokens;
  int T, V;
  int passes, bits;  // of a pass
  uint32_t* key[2];  // the last pass writes key[0] and at[0]
  int32_t* at[2];
  uint8_t* table;    // rows to zero, or NULL
  int64_t row_bytes;
};

struct SortShared {
  uint32_t hist[kSortWarps][kBins];
  uint32_t total[kBins], base[kBins], scan[kBins / 32];
  uint64_t held[kHeldCta];  // key and token, where a pass of the held sort puts them
};
struct FillShared {
  uint4 zeros[kZeroBytes / 16];
  uint8_t seen[kFillRows];
};

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// After the warps have counted their digits in hist: exclusive sums over the CTA's warps into hist, and
// over lower digits and the cluster's lower CTAs into base. A key's place is then base + hist + its
// rank among its warp's keys of the digit. Called by all threads, which may then read both.
template <int CL>
__device__ __forceinline__ void digit_places(SortShared& sh, int bins) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = threadIdx.x;
  const int rank = CL > 1 ? cluster_ctarank() : 0;
  __syncthreads();
  uint32_t mine = 0;
  if (d < bins) {
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = sh.hist[w][d];
      sh.hist[w][d] = mine;
      mine += c;
    }
    sh.total[d] = mine;
  }
  uint32_t all = mine, lower = 0;
  if (CL > 1) {
    cluster_sync();
    if (d < bins) {
      all = 0;
#pragma unroll
      for (int c = 0; c < CL; ++c) {
        const uint32_t v = ld_cluster(cluster_addr(&sh.total[d], c));
        if (c < rank) lower += v;
        all += v;
      }
    }
  }
  uint32_t inc = all;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  if (d < kBins && lane == 31) sh.scan[warp] = inc;
  __syncthreads();
  if (d < bins) {
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += sh.scan[w];
    sh.base[d] = before + inc - all + lower;
  }
  __syncthreads();
}

// Up to kHeld keys a thread, in registers through all passes: a pass ranks them as it counts them and puts
// them into shared memory (of the CTA that holds the place) for the next.
template <bool WIDE, int CL>
__device__ __forceinline__ void sort_held(const SortArgs& A, SortShared& sh) {
  const int rank = CL > 1 ? cluster_ctarank() : 0, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1;
  const int each = (A.T + CL * kSortThreads - 1) / (CL * kSortThreads);  // keys of a thread
  const int first = ((rank * kSortWarps + warp) * each) * 32 + lane;     // and its first, 32 apart
  const int cta_first = rank * kSortThreads * each;
  const int bins = 1 << A.bits;
  uint32_t key[kHeld], place[kHeld];
  int32_t at[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    at[j] = first + j * 32;
    key[j] = j < each && at[j] < A.T ? (uint32_t)id_of<WIDE>(A.tokens, at[j], A.V) : 0;
  }
  for (int pass = 0; pass < A.passes; ++pass) {
    const int shift = pass * A.bits;
    uint32_t* hist = sh.hist[warp];
    for (int d = lane; d < bins; d += 32) hist[d] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (j >= each) break;
      const bool live = first + j * 32 < A.T;
      const uint32_t d = live ? key[j] >> shift & (bins - 1) : kBins;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (live) place[j] = hist[d] + __popc(same & below);
      __syncwarp();
      if (live && !(same & below)) hist[d] += __popc(same);
      __syncwarp();
    }
    digit_places<CL>(sh, bins);
    const bool last = pass == A.passes - 1;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (j >= each || first + j * 32 >= A.T) break;
      const uint32_t d = key[j] >> shift & (bins - 1);
      const uint32_t to = place[j] + hist[d] + sh.base[d];
      const uint64_t held = (uint64_t)key[j] << 32 | (uint32_t)at[j];
      if (last) {
        A.key[0][to] = key[j];
        A.at[0][to] = at[j];
      } else if (CL == 1) {
        sh.held[to] = held;
      } else {
        const uint32_t span = kSortThreads * each, cta = to / span;
        st_cluster(cluster_addr(&sh.held[to - cta * span], cta), held);
      }
    }
    if (CL > 1) cluster_sync();  // after the last pass too: no CTA leaves while its totals are read
    else __syncthreads();
    if (last) break;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (j >= each) break;
      const uint64_t held = sh.held[first - cta_first + j * 32];
      key[j] = (uint32_t)(held >> 32);
      at[j] = (int32_t)held;
    }
    __syncthreads();
  }
}

// Any number of keys: read from global memory twice a pass, to count and to place them.
template <bool WIDE>
__device__ __forceinline__ void sort_any(const SortArgs& A, SortShared& sh) {
  const int rank = cluster_ctarank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1;
  // every warp of the cluster takes a run of tokens, in order of CTA and warp
  const int64_t each = ceil_div64(ceil_div64(A.T, kCluster * kSortWarps), 32) * 32;
  const int64_t first = min((rank * kSortWarps + warp) * each, (int64_t)A.T);
  const int64_t end = min(first + each, (int64_t)A.T);
  const int bins = 1 << A.bits;
  for (int pass = 0; pass < A.passes; ++pass) {
    const int shift = pass * A.bits, dst = (A.passes - 1 - pass) & 1;
    const uint32_t* from = A.key[dst ^ 1];
    const int32_t* from_at = A.at[dst ^ 1];
    auto key_of = [&](int64_t i) {
      return pass == 0 ? (uint32_t)id_of<WIDE>(A.tokens, i, A.V) : __ldcg(from + i);
    };
    uint32_t* hist = sh.hist[warp];
    for (int d = lane; d < bins; d += 32) hist[d] = 0;
    __syncwarp();
    for (int64_t i0 = first; i0 < end; i0 += 32) {
      const bool live = i0 + lane < end;
      const uint32_t d = live ? key_of(i0 + lane) >> shift & (bins - 1) : kBins;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (live && !(same & below)) hist[d] += __popc(same);
      __syncwarp();
    }
    digit_places<kCluster>(sh, bins);
    for (int64_t i0 = first; i0 < end; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool live = i < end;
      const uint32_t k = live ? key_of(i) : 0;
      const int32_t at = pass == 0 ? (int32_t)i : live ? __ldcg(from_at + i) : 0;
      const uint32_t d = live ? k >> shift & (bins - 1) : kBins;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      uint32_t place = 0;
      if (live) place = sh.base[d] + hist[d] + __popc(same & below);
      __syncwarp();
      if (live && !(same & below)) hist[d] += __popc(same);
      __syncwarp();
      if (live) {
        __stcg(A.key[dst] + place, k);
        __stcg(A.at[dst] + place, at);
      }
    }
    __threadfence();
    cluster_sync();  // all keys are where the next pass reads them, all totals have been read
  }
}

// Zeros into the rows of ids that do not occur: the CTA marks the ids of its rows that do, and every
// thread has the others' rows written by bulk copies from a buffer of zeros (6.3 TB/s; with a warp's
// stores row by row 4.1).
template <bool WIDE>
__device__ __forceinline__ void fill_zeros(const SortArgs& A, FillShared& sh, int cta, int ctas) {
  const int64_t r0 = (int64_t)A.V * cta / ctas, r1 = (int64_t)A.V * (cta + 1) / ctas;
  for (int i = threadIdx.x; i < kZeroBytes / 16; i += kSortThreads) sh.zeros[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  const uint32_t zeros = su32(sh.zeros);
  for (int64_t s0 = r0; s0 < r1; s0 += kFillRows) {
    const int rows = (int)min((int64_t)kFillRows, r1 - s0);
    for (int i = threadIdx.x; i < rows; i += kSortThreads) sh.seen[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < A.T; t += kSortThreads) {
      const int64_t i = id_of<WIDE>(A.tokens, t, A.V) - s0;
      if (i >= 0 && i < rows) sh.seen[i] = 1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows; i += kSortThreads) {
      if (sh.seen[i]) continue;
      uint8_t* row = A.table + (s0 + i) * A.row_bytes;
      for (int64_t b = 0; b < A.row_bytes; b += kZeroBytes) {
        const uint32_t n = (uint32_t)min((int64_t)kZeroBytes, A.row_bytes - b);
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(row + b), "r"(zeros), "r"(n)
                     : "memory");
      }
    }
    __syncthreads();
  }
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// CL: CTAs of the cluster that sorts, the grid's first. HELD: at most CL * kHeldCta tokens.
template <bool WIDE, int CL, bool HELD>
__global__ void __launch_bounds__(kSortThreads, 1) sort_fill_kernel(const __grid_constant__ SortArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= CL) fill_zeros<WIDE>(A, *(FillShared*)smem, blockIdx.x - CL, gridDim.x - CL);
  else if constexpr (HELD) sort_held<WIDE, CL>(A, *(SortShared*)smem);
  else sort_any<WIDE>(A, *(SortShared*)smem);
}

template <bool WIDE, int CL, bool HELD>
static moe_status_t sort_fill(const SortArgs& A, cudaStream_t s) {
  auto kern = sort_fill_kernel<WIDE, CL, HELD>;
  const size_t smem = std::max(sizeof(SortShared), sizeof(FillShared));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // clusters that the device holds at once (asked once a kernel and device): the SMs of a group are no
  // multiple of 8, and with a cluster more than fits the zeros took a second round
  static thread_local int known_dev = -1, clusters = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != known_dev) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return MOE_ERR_CUDA;
    clusters = num_sms();
    if (CL > 1 && cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess) return MOE_ERR_CUDA;
    known_dev = dev;
  }
  if (A.table) cfg.gridDim = dim3(std::max(2, clusters) * CL);  // the first one sorts, the others fill
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, A) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
template <bool WIDE>
static moe_status_t sort_fill(const SortArgs& A, cudaStream_t s) {
  // one CTA where that is as quick, or hidden behind the zeros (20 us for 8192 tokens, 140 MB of zeros): then
  // all other SMs write, not only those of whole clusters
  const bool hidden = A.T <= kHeldCta && A.table && A.V * A.row_bytes >= (int64_t)A.T * 16384;
  if (A.T <= kAloneUpTo || hidden) return sort_fill<WIDE, 1, true>(A, s);
  if (A.T <= kCluster * kHeldCta) return sort_fill<WIDE, kCluster, true>(A, s);
  return sort_fill<WIDE, kCluster, false>(A, s);
}

// ------------------------------------------------------------------- sums of runs
constexpr int kRun = 16;  // sorted rows of a warp: a lane keeps the id and the token of one

template <typename T, typename O>
struct RowPiece {  // the values of one 16-byte piece of T
  static constexpr int W = 16 / sizeof(T);
  // out (+)= scale * sum, rounded once
  static __device__ __forceinline__ void write(O* out, const float (&sum)[W], float scale, bool add) {
    float f[W];
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = sum[i] * scale;
    constexpr int PER = 16 / sizeof(O);
#pragma unroll
    for (int b = 0; b < W; b += PER) {
      float g[PER];
      uint4* p = (uint4*)(out + b);
      if (add) {
        Vec<O>::unpack(*p, g);
#pragma unroll
        for (int i = 0; i < PER; ++i) g[i] += f[b + i];
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) g[i] = f[b + i];
      }
      *p = Vec<O>::pack(g);
    }
  }
};

template <typename T, typename O>
__global__ void __launch_bounds__(256) run_sum_kernel(
    const uint4* __restrict__ dx, const uint32_t* __restrict__ keys, const int32_t* __restrict__ at,
    int n, int V, int vec, int slices, float scale, bool add, O* __restrict__ out,
    float* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  constexpr int W = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t c = item / slices;
  const int v = (int)(item % slices) * 32 + lane;
  const int64_t p0 = c * kRun;
  if (p0 >= n) return;
  const int rows = (int)min((int64_t)kRun, n - p0);
  const uint32_t key = lane < rows ? keys[p0 + lane] : V;
  const int32_t tok = lane < rows ? at[p0 + lane] : 0;
  const uint32_t before = p0 > 0 ? keys[p0 - 1] : 0xffffffffu;
  const uint32_t after = p0 + kRun < n ? keys[p0 + kRun] : 0xffffffffu;
  const bool mine = v < vec;
  const int64_t width = (int64_t)vec * W;
  float acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.f;
  bool from_before = true;  // the run began at the chunk's first row
  constexpr int AHEAD = 8;
  for (int i0 = 0; i0 < rows; i0 += AHEAD) {
    uint4 q[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const uint32_t k = __shfl_sync(0xffffffffu, key, i0 + j);
      const int t = __shfl_sync(0xffffffffu, tok, i0 + j);
      q[j] = make_uint4(0, 0, 0, 0);
      if (k < (uint32_t)V && mine) q[j] = __ldcs(dx + (int64_t)t * vec + v);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + j;
      const uint32_t k = __shfl_sync(0xffffffffu, key, i);
      if (k >= (uint32_t)V) return;  // sorted: no id from here on
      float f[W];
      Vec<T>::unpack(q[j], f);
#pragma unroll
      for (int e = 0; e < W; ++e) acc[e] += f[e];
      const bool last = i == kRun - 1;
      const uint32_t next = last ? after : __shfl_sync(0xffffffffu, key, (i + 1) & 31);
      if (!last && next == k) continue;
      // the run ends here, or goes on past the chunk
      const bool head = from_before && before == k, tail = last && next == k;
      if (mine) {
        if (!head && !tail) {
          RowPiece<T, O>::write(out + (int64_t)k * width + (int64_t)v * W, acc, scale, add);
        } else {
          float4* p = (float4*)(part + (2 * c + !head) * width + (int64_t)v * W);
#pragma unroll
          for (int e = 0; e < W; e += 4) p[e / 4] = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
        }
      }
#pragma unroll
      for (int e = 0; e < W; ++e) acc[e] = 0.f;
      from_before = false;
    }
  }
}

// Runs that cross chunks: the tail of the chunk in which they begin, then the heads of the ones that
// follow. A warp looks after one chunk's run in 128 columns; runs of many pieces are left to the
// whole CTA, whose warps take every eighth piece each.
constexpr int kAlone = 16;  // pieces that one warp adds by itself

template <typename O>
__device__ __forceinline__ void join_write(O* out, float4 s, float scale, bool add) {
  float f[4] = {s.x * scale, s.y * scale, s.z * scale, s.w * scale};
  if constexpr (sizeof(O) == 4) {
    float4* p = (float4*)out;
    if (add) {
      const float4 o = *p;
      f[0] += o.x; f[1] += o.y; f[2] += o.z; f[3] += o.w;
    }
    *p = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    uint2* p = (uint2*)out;
    if (add) {
      const uint2 o = *p;
      f[0] += __uint_as_float(o.x << 16); f[1] += __uint_as_float(o.x & 0xFFFF0000u);
      f[2] += __uint_as_float(o.y << 16); f[3] += __uint_as_float(o.y & 0xFFFF0000u);
    }
    *p = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
  }
}

template <typename O>
__global__ void __launch_bounds__(256) join_kernel(const uint32_t* __restrict__ keys, int n, int V,
                                                   int H, int columns, float scale, bool add,
                                                   const float* __restrict__ part,
                                                   O* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  __shared__ int count[8];
  __shared__ float4 sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t group = blockIdx.x / columns;
  const int col = (int)(blockIdx.x % columns) * 128 + lane * 4;
  const int64_t chunks = ceil_div64(n, kRun), c = group * 8 + warp;
  // the run of the chunk's last row, if it begins in this chunk and goes on: its pieces
  int pieces = 0;
  uint32_t key = 0;
  if (c + 1 < chunks) {
    key = keys[c * kRun + kRun - 1];
    const bool whole = keys[c * kRun] == key && c > 0 && keys[c * kRun - 1] == key;
    if (key < (uint32_t)V && !whole) {
      int64_t j = c + 1;
      for (;; j += 32) {
        const bool on = j + lane < chunks && keys[(j + lane) * kRun] == key;
        const uint32_t run = __ballot_sync(0xffffffffu, on);
        if (run != 0xffffffffu) {
          j += __ffs(~run) - 1;
          break;
        }
      }
      pieces = (int)(j - c);
      if (pieces == 1) pieces = 0;  // goes no further
    }
  }
  auto piece = [&](int64_t at, int i) {  // piece i of the run that begins in chunk `at`
    return col < H ? *(const float4*)(part + (2 * (at + i) + (i == 0)) * H + col) : make_float4(0, 0, 0, 0);
  };
  auto plus = [](float4& a, const float4& b) { a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w; };
  if (pieces && pieces <= kAlone) {
    float4 s = piece(c, 0);
#pragma unroll 8
    for (int i = 1; i < pieces; ++i) plus(s, piece(c, i));
    if (col < H) join_write(out + (int64_t)key * H + col, s, scale, add);
  }
  if (lane == 0) count[warp] = pieces > kAlone ? pieces : 0;
  __syncthreads();
  for (int w = 0; w < 8; ++w) {
    const int m = count[w];
    if (!m) continue;
    const int64_t at = group * 8 + w;
    float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 8
    for (int i = warp; i < m; i += 8) plus(s, piece(at, i));
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < H) {
      s = sums[0][lane];
#pragma unroll
      for (int i = 1; i < 8; ++i) plus(s, sums[i][lane]);
      join_write(out + (int64_t)keys[at * kRun + kRun - 1] * H + col, s, scale, add);
    }
    __syncthreads();
  }
}

// Workspace: two (key, token) arrays for the passes, then the partial sums.
struct Layout {
  size_t key[2], at[2], part, total;
};
static Layout layout(int T, int H) {
  Layout l{};
  const size_t n = align_up((size_t)T * 4, 256);
  l.key[0] = 0;
  l.key[1] = n;
  l.at[0] = 2 * n;
  l.at[1] = 3 * n;
  l.part = 4 * n;
  const size_t chunks = ceil_div(T, kRun);
  l.total = l.part + (chunks > 1 ? chunks * 2 * H * sizeof(float) : 0);
  return l;
}

}  // namespace embedding

using namespace embedding;
using ebf = __nv_bfloat16;

moe_status_t launch_embed(const void* tokens, bool wide, int T, const void* table, int V, int H,
                          moe_dtype_t dt, float scale, void* out, cudaStream_t s) {
  const int vec = (int)((size_t)H * dtype_size(dt) / 16);
  auto go = [&](auto kern, int pieces) {
    const int parts = ceil_div(vec, 32 * pieces);
    const int64_t most = std::max(1, num_sms() * 32 / parts);  // CTAs along the tokens
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div64(T, 8), most), parts);
    return launch_k(kern, grid, dim3(256), 0, s, tokens, T, (const uint4*)table, V, vec, scale, (uint4*)out);
  };
  const bool few = (int64_t)T * vec < (int64_t)num_sms() * 2048;  // a piece a thread fills no SM twice
  if (dt == MOE_BF16) {
    if (few) return wide ? go(embed_kernel<ebf, true, 1>, 1) : go(embed_kernel<ebf, false, 1>, 1);
    return wide ? go(embed_kernel<ebf, true, 4>, 4) : go(embed_kernel<ebf, false, 4>, 4);
  }
  if (few) return wide ? go(embed_kernel<float, true, 1>, 1) : go(embed_kernel<float, false, 1>, 1);
  return wide ? go(embed_kernel<float, true, 4>, 4) : go(embed_kernel<float, false, 4>, 4);
}

size_t embed_ws_bytes(int T, int V, int H) { return layout(T, H).total; }

moe_status_t launch_embed_backward(const void* dx, const void* tokens, bool wide, int T, int V, int H,
                                   moe_dtype_t dt, moe_dtype_t out_dt, float scale, int accumulate,
                                   void* dtable, void* ws, cudaStream_t s) {
  const int vec = (int)((size_t)H * dtype_size(dt) / 16), slices = ceil_div(vec, 32);
  const int chunks = ceil_div(T, kRun);
  const int64_t blocks = ceil_div64((int64_t)chunks * slices, 8);
  const int columns = ceil_div(H, 128);
  const int64_t joins = (int64_t)ceil_div(chunks, 8) * columns;
  if (blocks > 0x7fffffff || joins > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  const Layout l = layout(T, H);
  uint8_t* w = (uint8_t*)ws;
  SortArgs A{};
  A.tokens = tokens;
  A.T = T;
  A.V = V;
  int bits = 1;  // of the keys 0 to V
  while (bits < 31 && (V >> bits)) ++bits;
  A.passes = ceil_div(bits, kDigit);
  A.bits = ceil_div(bits, A.passes);
  for (int i = 0; i < 2; ++i) {
    A.key[i] = (uint32_t*)(w + l.key[i]);
    A.at[i] = (int32_t*)(w + l.at[i]);
  }
  A.table = accumulate ? nullptr : (uint8_t*)dtable;
  A.row_bytes = (int64_t)H * dtype_size(out_dt);
  moe_status_t st = wide ? sort_fill<true>(A, s) : sort_fill<false>(A, s);
  if (st != MOE_OK) return st;
  const uint32_t* keys = A.key[0];
  const int32_t* at = A.at[0];
  float* part = (float*)(w + l.part);
  const bool add = accumulate != 0;
  auto sums = [&](auto run, auto join, auto* out) {
    const moe_status_t r = launch_k(run, dim3((unsigned)blocks), dim3(256), 0, s, (const uint4*)dx, keys, at, T,
                                    V, vec, slices, scale, add, out, part);
    if (r != MOE_OK || chunks == 1) return r;
    return launch_k(join, dim3((unsigned)joins), dim3(256), 0, s, keys, T, V, H, columns, scale, add,
                    (const float*)part, out);
  };
  if (dt == MOE_F32) return sums(run_sum_kernel<float, float>, join_kernel<float>, (float*)dtable);
  if (out_dt == MOE_F32) return sums(run_sum_kernel<ebf, float>, join_kernel<float>, (float*)dtable);
  return sums(run_sum_kernel<ebf, ebf>, join_kernel<ebf>, (ebf*)dtable);
}

}  // namespace moe
