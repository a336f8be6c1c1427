// experts_tc.cu — the experts' bf16 products and weight gradients on CTA pairs
// (tcgen05.mma.cta_group::2, M = 256, N = 256, fp32 accumulators in tensor memory).
//
// Five products over the rows of each expert (P rows, run of expert e at start[e], cnt[e] of them):
//   up         D = xs W13[e]^T   rows x (gate | up): an N = 256 tile is 128 gate and the same 128 up
//                                columns, so the epilogue holds both halves of the SwiGLU
//   down       D = act W2[e]^T
//   down_grad  D = dys W2[e]     then the SwiGLU's gradient from the stored pre-activations
//   up_grad    D = dh13 W13[e]
//   weight     D = dy_e^T a_e    reduction over the expert's rows
// The tensor cores read a shared-memory operand with either of its two axes contiguous, so the
// gradients need no transposed copies: a weight read the other way round (down_grad, up_grad) and
// both operands of the weight gradient are loaded as 64-column boxes, 128 bytes a row, and given
// to the MMA as M/N-major tiles. Padding each expert's run to 16 rows (one MMA K step) with zeros
// makes the weight gradient's reduction exact without masks.
//
// Shared memory is what bounds the products: per MMA an SM reads 8 KB of operands from it in 128
// clocks at the full tensor rate, while the TMA writes 64 bytes a clock into it (48 with wide items,
// below), of 128 bytes a clock in all. So the epilogue keeps out of it: a thread holds one row of a
// tile and stores (and, in down_grad, loads) whole 32-byte sectors of it directly. Measured with
// 1024 rows an expert, tiles staged through shared memory for full lines took 5 % longer with wide
// items on and off, whether the TMA or the threads stored them. (The weight gradients' narrow form,
// whose reductions are short and results large, is the exception: see there.)
//
// The accumulators cut sums off where fp32 arithmetic rounds: the error is toward zero and grows with the
// length of a reduction (weight gradients of random rows: 4.7e-7 of their size over 512 rows, 2.1e-6 over 2048,
// 9.1e-6 over 8192, the same as in the library's bf16 product with fp32 results). bf16 results, off by 1.7e-3
// from their rounding, do not show it. fp32 weight gradients leave the accumulators every 512 rows and are
// added up in registers: 4.8e-7 over 8192 rows. That takes 2 to 3 % at up to 1000 rows an expert, 5 % at
// 2048, 7 % at 4096, and the wide form (below), whose two tiles would be 256 sums a thread: with it, 2 experts of
// 4096 x 4096 over 8192 rows took 343 us, without 387.
//
// Roles in each CTA of a pair: warp 0 issues the TMA loads into a ring of stages, warp 1 of the
// leader issues the MMAs, the others are the epilogue. Tensor memory holds two 256-column
// accumulators. Work items are (expert, 256-row tile, NH 256-column tiles), weight panels outermost
// within an expert, so that pairs running together share them in L2; persistent CTA pairs take them
// in turn. All waits are bounded (status kStatusTimeout, no trap).
//
// NH = 2: both accumulators belong to one item, which reads each A tile once for 512 columns, a
// quarter fewer operand bytes a product; those bytes, not the MMAs, bound the NH = 1 form (with
// operands of zeros, where power does not count, it ran at 0.67 of the tensor rate whether the ring
// had 4, 5 or 6 stages). The accumulators are not double-buffered then, so the order of the MMAs hides
// the epilogue: the first accumulator gets the last stages of an item first, and is drained while
// the second gets them; an item's first stages go to the first accumulator while the second is
// still being drained. NH = 1 (the accumulators alternate between items) takes over where the wide
// items would leave pairs without work.
#include "tc_ptx.cuh"
#include "train.cuh"

namespace moe {
namespace etc {

using namespace ptx;

__device__ int g_status;

enum Kind { kKUp = 0, kKDown = 1, kKDownGrad = 2, kKUpGrad = 3, kKWeight32 = 4, kKWeight16 = 5 };

constexpr int kTmemCols = 512;
constexpr int A_BYTES = 128 * 128;
constexpr int B_BYTES = 128 * 128;   // of one 256-column tile
constexpr int CHUNK = 64 * 128;      // one 64-column box of an M/N-major operand: 64 K rows x 128 B

constexpr int OUT_BYTES = 32 * 128;  // a staged tile of dW: 32 rows of 128 bytes
constexpr int kSplit = 8;            // stages (of BK rows) of an fp32 dW that the accumulators add up

template <int KIND>
struct Traits {
  static constexpr bool weight = KIND >= kKWeight32;
  static constexpr bool a_mn = weight;  // operand contiguous along M rather than K
  static constexpr bool b_mn = KIND >= kKDownGrad;
  static constexpr bool split = KIND == kKWeight32;  // sums leave the accumulators every kSplit stages
  static constexpr uint32_t idesc =
      idesc_bf16(256, 256) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
};

template <int KIND, int NH>
struct Layout {
  static constexpr bool staged = Traits<KIND>::weight && NH == 1;  // dW leaves through the TMA
  static constexpr int kStages = NH == 2 ? 4 : staged ? 5 : 6;
  static constexpr int kEpiWarps = 8;  // two a 32-lane quarter of tensor memory
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kStageB = NH * B_BYTES;
  static constexpr size_t a = 0;
  static constexpr size_t b = a + (size_t)kStages * A_BYTES;
  static constexpr size_t out = b + (size_t)kStages * kStageB;
  static constexpr size_t bars = out + (staged ? (size_t)kEpiWarps * OUT_BYTES : 0);
  static constexpr size_t misc = bars + (2 * kStages + 5) * 8;
  static constexpr size_t start = misc + 16;
  static constexpr size_t cnt = start + (kMaxExperts + 1) * 4;
  static constexpr size_t pre = cnt + kMaxExperts * 4;
  static constexpr size_t end = pre + (kMaxExperts + 1) * 4;
  static constexpr size_t bytes = 1024 + end;
};
static_assert(Layout<kKUp, 1>::bytes <= 232448 && Layout<kKUp, 2>::bytes <= 232448 &&
                  Layout<kKWeight32, 1>::bytes <= 232448, "shared memory");

struct Params {
  const int32_t* counts;
  const float* h13;  // down_grad: the pre-activations [rows, 2I]
  void* out;
  void* act;         // up, down_grad
  int E, rows;
  int M;             // weight: rows of dW[e]
  int N;             // columns of the result (up: I)
  int K;             // reduction (rows kinds)
  int m_tiles, n_tiles;  // n_tiles: 256-column tiles (up: 128 gate and up columns)
  int n_items;           // column items: NH tiles each
  int accumulate;
  int out_bytes, act_bytes;  // bytes of a row of out and act
  int wide;                  // whether all of their rows start on 32-byte boundaries
};

struct Maps {
  CUtensorMap a, b0, b1;
  CUtensorMap a16, b16;  // weight: 16-row boxes, for the end of a reduction
  CUtensorMap o;         // weight: dW in 32-row boxes of 128 bytes
};

// M/N-major operand tile: 128-byte swizzled rows of 64 elements along M or N, one row a K index;
// 8-row groups 1024 bytes apart along K (stride offset), 64-element chunks CHUNK bytes apart along
// M or N (leading offset). Sixteen K rows further is 2048 bytes further.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(CHUNK >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void store_3d(const CUtensorMap* tm, const void* src, int c0, int c1,
                                         int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          (uint64_t)tm),
      "r"(c0), "r"(c1), "r"(c2), "r"(su32(src))
      : "memory");
}
__device__ __forceinline__ void add_3d(const CUtensorMap* tm, const void* src, int c0, int c1,
                                       int c2) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], "
      "[%4];" ::"l"((uint64_t)tm),
      "r"(c0), "r"(c1), "r"(c2), "r"(su32(src))
      : "memory");
}
// The 16-byte piece c of row r of a staged tile (128-byte swizzle, as its map has it).
__device__ __forceinline__ uint4* piece(uint8_t* tile, int r, int c) {
  return reinterpret_cast<uint4*>(tile + r * 128 + ((c ^ (r & 7)) << 4));
}
// Whether a phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(su32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}

// An arrival on CTA `rank`'s barrier that orders none of this thread's own reads and writes. It hands an
// accumulator back, whose reads tcgen05.wait::ld has seen finished and tcgen05.fence orders; an
// arrival with release would also wait for the tile's stores to be acknowledged (1650 clocks of the 4200 of
// a 256 x 256 tile of bf16 dW: 64 experts of 4096 x 2048 over 8 rows each 243 -> 184 us).
__device__ __forceinline__ void arrive_relaxed(uint64_t* b, uint32_t rank) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(b, rank))
               : "memory");
}

// Thirty-two bytes of a row, to or from global memory: one instruction where `wide` (every row of the
// matrix starts on a 32-byte boundary), else two. n: 16-byte pieces left of the row's end.
__device__ __forceinline__ void put32(void* p, const uint32_t (&v)[8], bool wide, int n) {
  if (wide) {
    if (n > 0)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                   "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                   : "memory");
  } else {
    if (n > 0) ((uint4*)p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    if (n > 1) ((uint4*)p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void get32(const void* p, uint32_t (&v)[8], bool wide, int n) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0;
  if (wide) {
    if (n > 0)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                     "=r"(v[6]), "=r"(v[7])
                   : "l"(p)
                   : "memory");
  } else {
    if (n > 0) {
      const uint4 x = ((const uint4*)p)[0];
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
    if (n > 1) {
      const uint4 x = ((const uint4*)p)[1];
      v[4] = x.x; v[5] = x.y; v[6] = x.z; v[7] = x.w;
    }
  }
}
// Sixteen fp32 values of a row, or thirty-two bf16 ones as pairs: two 32-byte pieces at p.
__device__ __forceinline__ void put64(void* p, const uint32_t* v, bool wide, int n) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[8 * h + i];
    put32((uint8_t*)p + 32 * h, x, wide, n - 2 * h);
  }
}

// Thirty-two fp32 values plus the bf16 ones at p, in fp32: the sum is rounded once.
__device__ __forceinline__ void add_old(uint32_t (&v)[32], const uint8_t* p, bool wide, int n) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t o[8];
    get32(p + 32 * i, o, wide, n - 2 * i);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int x = 16 * i + 2 * j;
      v[x] = __float_as_uint(__uint_as_float(v[x]) + __uint_as_float(o[j] << 16));
      v[x + 1] = __float_as_uint(__uint_as_float(v[x + 1]) + __uint_as_float(o[j] & 0xFFFF0000u));
    }
  }
}

// The hardware's exponential and reciprocal: results are rounded to bf16, and the epilogue has to keep up
// with the tensor cores. The exponential is off by up to 2 + 1.2 |v| units of fp32's last place, a hundred
// at the end of its range: 1/300 of bf16's half step. Below v = -87 the quotient is 0.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

struct Item {
  int e, n, nh;    // expert, first column tile, column tiles
  int m0;          // first row of the tile (weight: first row of dW[e])
  int row0, cnt;   // the expert's rows
  int num_kb;
  bool live1;      // the peer's half of the tile holds rows
};

template <int KIND, int NH>
__device__ __forceinline__ Item item_of(int w, const Params& P, const int* start, const int* cnt,
                                        const int* pre) {
  Item it;
  int n;
  if (Traits<KIND>::weight) {
    const int per = P.m_tiles * P.n_items;
    it.e = w / per;
    const int rest = w - it.e * per;
    n = rest % P.n_items;
    it.m0 = rest / P.n_items * 256;
    it.row0 = start[it.e];
    it.cnt = cnt[it.e];
    it.num_kb = (it.cnt + BK - 1) / BK;
    it.live1 = true;
  } else {
    int lo = 0, hi = P.E - 1;  // the last expert whose first item is at or before w
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * P.n_items <= w) lo = mid; else hi = mid - 1;
    }
    const int c = pre[lo + 1] - pre[lo];
    const int local = w - pre[lo] * P.n_items;
    it.e = lo;
    n = local / c;
    const int i = local - n * c;
    it.row0 = start[lo];
    it.cnt = cnt[lo];
    it.m0 = it.row0 + i * 256;
    it.num_kb = (P.K + BK - 1) / BK;
    it.live1 = i * 256 + 128 < it.cnt;
  }
  it.n = n * NH;
  it.nh = min(NH, P.n_tiles - it.n);
  return it;
}

template <int KIND, int NH>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<KIND, NH>::kThreads, 1)
    expert_pair_kernel(const __grid_constant__ Maps TM, const Params P) {
  using R = Traits<KIND>;
  using LY = Layout<KIND, NH>;
  constexpr int kStages = LY::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sA = smem + LY::a;
  uint8_t* sB = smem + LY::b;
  uint64_t* full = (uint64_t*)(smem + LY::bars);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // per accumulator
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = (uint32_t*)(smem + LY::misc);
  volatile int* abort_flag = (volatile int*)(smem + LY::misc + 4);
  int* start = (int*)(smem + LY::start);
  int* cnt = (int*)(smem + LY::cnt);
  int* pre = (int*)(smem + LY::pre);
  int* status = &g_status;

  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);  // the leader's counts both CTAs' bytes
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * LY::kEpiWarps);  // both CTAs' epilogue warps (the leader's is used)
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
    prefetch_tmap(&TM.a);
    prefetch_tmap(&TM.b0);
  }
  if (warp == 1) {
    tmem_alloc<2>(tmem_slot, kTmemCols);
    tmem_relinquish<2>();
    tc_fence_before();
  }
  cluster_sync();  // barriers initialised and tensor memory allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  bool mismatch = false;
  if (threadIdx.x == 0) {  // the leader's MMAs write the peer's rows at the leader's address
    uint32_t peer, other;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(su32(tmem_slot)), "r"(rank ^ 1u));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(peer) : "memory");
    if (other != tmem_base) {
      *abort_flag = 1;
      mismatch = true;
    }
  }

  pdl_wait();  // global memory is touched only past this point
  if (mismatch) atomicExch(status, kStatusPairTmem);
  load_counts(P.counts, P.E, cnt);
  __syncthreads();
  if (warp == 0) {
    expert_rows(P.E, P.rows, start, cnt, blockIdx.x == 0 ? status : nullptr);
    __syncwarp();
    if (!R::weight) {  // pre[e]: 256-row tiles of lower experts
      int base = 0;
      for (int e0 = 0; e0 < P.E; e0 += 32) {
        const int e = e0 + lane;
        const int c = e < P.E ? (cnt[e] + 255) / 256 : 0;
        int inc = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, inc, off);
          if (lane >= off) inc += o;
        }
        if (e < P.E) pre[e] = base + inc - c;
        base += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) pre[P.E] = base;
    }
  }
  __syncthreads();
  const int total = R::weight ? P.E * P.m_tiles * P.n_items : pre[P.E] * P.n_items;
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int w = pair; w < total && ok; w += num_pairs) {
        const Item it = item_of<KIND, NH>(w, P, start, cnt, pre);
        const uint32_t row_bytes = 2u * (A_BYTES + it.nh * B_BYTES) - (it.live1 ? 0u : (uint32_t)A_BYTES);
        for (int kb = 0; kb < it.num_kb; ++kb) {
          if (!wait_bounded(&empty[s], phase ^ 1u, abort_flag, status)) {
            ok = false;
            break;
          }
          const uint32_t fl = cluster_addr(&full[s], 0);
          uint8_t* a = sA + s * A_BYTES;
          uint8_t* b = sB + s * LY::kStageB;
          if (R::weight) {
            // the last stage of the reduction: as many 16-row steps as it has (298 -> 289 us when it came, for
            // dW of 32 experts of 5760 x 2880 over 1 to 8 rows each, 189 us now)
            const int left = it.cnt - kb * BK, steps = left > 48 ? 4 : (left + 15) / 16;
            if (leader) mbar_expect_tx(&full[s], 2u * (1 + it.nh) * (steps * 4096u));
            const int y = it.row0 + kb * BK, m = it.m0 + (int)rank * 128;
            auto two = [&](uint8_t* to, const CUtensorMap* whole, const CUtensorMap* part, int x) {
              if (steps == 4) {
                tma_2d_pair(to, whole, fl, x, y);
                tma_2d_pair(to + CHUNK, whole, fl, x + 64, y);
              } else {
                for (int j = 0; j < steps; ++j) {
                  tma_2d_pair(to + j * 2048, part, fl, x, y + 16 * j);
                  tma_2d_pair(to + CHUNK + j * 2048, part, fl, x + 64, y + 16 * j);
                }
              }
            };
            two(a, &TM.a, &TM.a16, m);
            for (int h = 0; h < it.nh; ++h, b += B_BYTES)
              two(b, &TM.b0, &TM.b16, (it.n + h) * 256 + (int)rank * 128);
          } else {
            if (leader) mbar_expect_tx(&full[s], row_bytes);
            // the peer's rows of a half-filled tile are neither loaded nor stored
            if (leader || it.live1) tma_2d_pair(a, &TM.a, fl, kb * BK, it.m0 + (int)rank * 128);
            for (int h = 0; h < it.nh; ++h, b += B_BYTES) {
              const int n = it.n + h;
              if (KIND == kKUp) {  // leader: gate rows, peer: the same up rows
                tma_3d_pair(b, rank ? &TM.b1 : &TM.b0, fl, kb * BK, n * 128, it.e);
              } else if (KIND == kKDown) {
                tma_3d_pair(b, &TM.b0, fl, kb * BK, n * 256 + (int)rank * 128, it.e);
              } else {
                const int c = n * 256 + (int)rank * 128;
                tma_3d_pair(b, &TM.b0, fl, c, kb * BK, it.e);
                tma_3d_pair(b + CHUNK, &TM.b0, fl, c + 64, kb * BK, it.e);
              }
            }
          }
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ leader: MMA issuer
    if (leader && lane == 0) {
      // stages are counted: stage number g sits in slot g % kStages; acc_phase bit a is the phase
      // of accumulator a
      int g0 = 0, acc = 0;
      uint32_t acc_phase = 0;
      bool issued = false, ok = true;
      for (int w = pair; w < total && ok; w += num_pairs) {
        const Item it = item_of<KIND, NH>(w, P, start, cnt, pre);
        const int T = it.num_kb;
        if (T == 0) continue;
        const int K = R::weight ? it.cnt : P.K;
        auto wait_full = [&](int kb) {
          const int g = g0 + kb;
          if (!wait_bounded(&full[g % kStages], (uint32_t)(g / kStages) & 1u, abort_flag, status))
            return false;
          tc_fence_after();
          return true;
        };
        // stage kb into accumulator a, B tile h; stage `first` overwrites it
        auto mma = [&](int kb, int h, int a, int first = 0) {
          const int s = (g0 + kb) % kStages;
          const uint32_t sa = su32(sA + s * A_BYTES), sb = su32(sB + s * LY::kStageB + h * B_BYTES);
          const uint32_t d = tmem_base + (uint32_t)(a * 256);
          const int steps = min(BK / UMMA_K, (K - kb * BK + UMMA_K - 1) / UMMA_K);
#pragma unroll
          for (int kk = 0; kk < BK / UMMA_K; ++kk) {
            if (kk < steps)
              umma_bf16<2>(d, R::a_mn ? mn_desc(sa + kk * 2048) : sw128_desc(sa + kk * 32),
                           R::b_mn ? mn_desc(sb + kk * 2048) : sw128_desc(sb + kk * 32), R::idesc,
                           ((kb - first) | kk) != 0 ? 1u : 0u);
          }
          issued = true;
        };
        auto release = [&](int kb) { umma_commit_pair(&empty[(g0 + kb) % kStages], 0x3); };
        auto acc_free = [&](int a) {
          if (!wait_bounded(&tempty[a], ((acc_phase >> a) & 1u) ^ 1u, abort_flag, status)) return false;
          tc_fence_after();
          return *abort_flag == 0;
        };
        if constexpr (R::split) {
          for (int k0 = 0; k0 < T && ok; k0 += kSplit) {
            const int a = acc, k1 = min(T, k0 + kSplit);
            if (!(ok = acc_free(a))) break;
            for (int kb = k0; kb < k1; ++kb) {
              if (!(ok = wait_full(kb))) break;
              mma(kb, 0, a, k0);
              release(kb);
            }
            if (!ok) break;
            umma_commit_pair(&tfull[a], 0x3);
            acc_phase ^= 1u << a;
            acc ^= 1;
          }
          if (!ok) break;
        } else if (NH == 1 || it.nh == 1) {
          const int a = NH == 1 ? acc : 0;
          if (!acc_free(a)) break;
          for (int kb = 0; kb < T && ok; ++kb) {
            if (!(ok = wait_full(kb))) break;
            mma(kb, 0, a);
            release(kb);
          }
          if (!ok) break;
          umma_commit_pair(&tfull[a], 0x3);
          acc_phase ^= 1u << a;
          if (NH == 1) acc ^= 1;
        } else {
          if (!acc_free(0)) break;
          // the first stages for accumulator 0 alone, while 1 is still being drained
          int p = 0;
          while (p < min(kStages, T) && ok && !mbar_test(&tempty[1], ((acc_phase >> 1) & 1u) ^ 1u)) {
            if (!(ok = wait_full(p))) break;
            mma(p++, 0, 0);
          }
          if (!ok || !acc_free(1)) break;
          if (p == T) umma_commit_pair(&tfull[0], 0x3);
          int r = 0;
          for (; r < p; ++r) {
            mma(r, 1, 1);
            release(r);
          }
          for (; p < T - kStages && ok; ++p, ++r) {
            if (!(ok = wait_full(p))) break;
            mma(p, 0, 0);
            mma(p, 1, 1);
            release(p);
          }
          if (!ok) break;
          // the last stages: all of them for accumulator 0, which its epilogue then drains
          if (p < T) {
            for (; p < T && ok; ++p) {
              if (!(ok = wait_full(p))) break;
              mma(p, 0, 0);
            }
            if (!ok) break;
            umma_commit_pair(&tfull[0], 0x3);
            for (; r < T; ++r) {
              mma(r, 1, 1);
              release(r);
            }
          }
          umma_commit_pair(&tfull[1], 0x3);
          acc_phase ^= 3u;
        }
        g0 += T;
      }
      if (issued) {  // every MMA of this thread finished before tensor memory is freed
        umma_commit<2>(drain);
        wait_bounded(drain, 0, abort_flag, status);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                 // tensor-memory lanes q*32 .. q*32+31
    const int part = (warp - 2) >> 2;       // which half of a tile's columns
    constexpr int kCols = 256 / (LY::kEpiWarps / 4);
    if (!R::weight) {  // rows past the last run are zeroed while the first tile is computed
      const int t = (warp - 2) * 32 + lane;
      const uint4 z = make_uint4(0, 0, 0, 0);
      for (int p = start[P.E] + (int)blockIdx.x; p < P.rows; p += gridDim.x) {
        for (int v = t; v < P.out_bytes / 16; v += 32 * LY::kEpiWarps)
          ((uint4*)((uint8_t*)P.out + (int64_t)p * P.out_bytes))[v] = z;
        for (int v = t; v < P.act_bytes / 16; v += 32 * LY::kEpiWarps)
          ((uint4*)((uint8_t*)P.act + (int64_t)p * P.act_bytes))[v] = z;
      }
    }
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok_all = true;
    for (int w = pair; w < total && ok_all; w += num_pairs) {
      const Item it = item_of<KIND, NH>(w, P, start, cnt, pre);
      if (R::weight && it.num_kb == 0 && P.accumulate) continue;
      const bool computed = it.num_kb != 0;
      const int m = it.m0 + (int)rank * 128 + q * 32;  // first row of this warp's 32
      // this thread's row: whether it is stored (rows kinds: up to the run's padded end, zeros past cnt)
      const int end = R::weight ? P.M : min(it.row0 + (it.cnt + kRowBlock - 1) / kRowBlock * kRowBlock, P.rows);
      const bool store = m + lane < end;
      const bool slot = R::weight ? computed : m + lane < it.row0 + it.cnt;
      uint8_t* const out = (uint8_t*)P.out + ((R::weight ? (int64_t)it.e * P.M : 0) + m + lane) * P.out_bytes;
      uint8_t* const act = (uint8_t*)P.act + (int64_t)(m + lane) * P.act_bytes;
      const float* const hrow = P.h13 + (int64_t)(m + lane) * 2 * P.N;
      const bool wide = P.wide;
      if constexpr (R::split) {
        // fp32 dW: the sums of kSplit stages at a time are added up in registers; the last ones are added on
        // their way out, as whole 128-byte lines through the TMA, which also clips ragged edges and adds to
        // fp32. dW of 64 experts of 4096 x 2048 over 8 rows each took 339 us (6.3 TB/s) so, 444 in stores from
        // registers; a second buffer a warp, for a stage of the ring less, or sixteen warps of one 359 and 361.
        float sum[kCols] = {};
        const int n0 = it.n * 256 + part * kCols;
        const int segs = (it.num_kb + kSplit - 1) / kSplit;
        uint8_t* const t = smem + LY::out + (size_t)(warp - 2) * OUT_BYTES;
        uint32_t tb = 0;
#pragma unroll 1
        for (int g = 0; g < segs; ++g) {
          int ok = 1;
          if (lane == 0) ok = wait_bounded_inline(&tfull[acc], (acc_phase >> acc) & 1u, abort_flag, status);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) {
            ok_all = false;
            break;
          }
          tc_fence_after();
          tb = tmem_base + (uint32_t)(acc * 256 + part * kCols) + ((uint32_t)(q * 32) << 16);
          if (g == segs - 1) break;
          if (m < end) {
#pragma unroll
            for (int c = 0; c < kCols / 16; ++c) {  // sixteen at a time: 128 sums leave no more registers
              if (n0 + 16 * c >= P.N) break;
              uint32_t v[16];
              tmem_ld16(tb + 16 * c, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[16 * c + i] += __uint_as_float(v[i]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_relaxed(&tempty[acc], 0);
          acc_phase ^= 1u << acc;
          acc ^= 1;
        }
        if (ok_all && m < end) {
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            const int col = n0 + 32 * c;
            if (col >= P.N) break;
            // the tile's last store has been read
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 32; x += 16) {
              uint32_t v[16] = {};
              if (segs) {
                tmem_ld16(tb + 32 * c + x, v);
                tmem_ld_wait();
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float* f = &sum[32 * c + x + 4 * i];
                *piece(t, lane, x / 4 + i) = make_uint4(
                    __float_as_uint(f[0] + __uint_as_float(v[4 * i])), __float_as_uint(f[1] + __uint_as_float(v[4 * i + 1])),
                    __float_as_uint(f[2] + __uint_as_float(v[4 * i + 2])), __float_as_uint(f[3] + __uint_as_float(v[4 * i + 3])));
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (P.accumulate) add_3d(&TM.o, t, col, m, it.e);
              else store_3d(&TM.o, t, col, m, it.e);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          }
        }
        if (segs && ok_all) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_relaxed(&tempty[acc], 0);
          acc_phase ^= 1u << acc;
          acc ^= 1;
        }
      }
      for (int h = 0; !R::split && h < it.nh; ++h) {
        const int a = NH == 1 ? acc : h;
        const int n = it.n + h;
        // 16-byte pieces of a row of es-byte values that lie left of column N
        auto left = [&](int col, int es) { return (P.N - col) * es / 16; };
        uint32_t gq[4][8], uq[4][8];  // down_grad: pre-activations, asked for before they are needed
        auto ask = [&](int col) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = slot ? left(col + 8 * i, 4) : 0;
            get32(hrow + col + 8 * i, gq[i], wide, k);
            get32(hrow + P.N + col + 8 * i, uq[i], wide, k);
          }
        };
        if (KIND == kKDownGrad) ask(n * 256 + part * kCols);
        if (computed) {
          int ok = 1;
          if (lane == 0) ok = wait_bounded(&tfull[a], (acc_phase >> a) & 1u, abort_flag, status);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) {
            ok_all = false;
            break;
          }
          tc_fence_after();
        }
        const uint32_t tb = tmem_base + (uint32_t)(a * 256) + ((uint32_t)(q * 32) << 16);
        const bool some = m < end;  // of the warp
        if (some && KIND == kKUp) {
          const int n0 = n * 128;
#pragma unroll 1
          for (int c = part * (kCols / 2); c < (part + 1) * (kCols / 2); c += 32) {
            const int col = n0 + c;
            if (col >= P.N) break;
            __syncwarp();
            uint32_t g32[32], u32[32], ap[16];
            tmem_ld32(tb + c, g32);
            tmem_ld32(tb + 128 + c, u32);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float a2[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int j = 2 * i + y;
                if (!slot) g32[j] = u32[j] = 0;
                const float g = __uint_as_float(g32[j]);
                a2[y] = g * sigmoid(g) * __uint_as_float(u32[j]);
              }
              ap[i] = pack_bf16(a2[0], a2[1]);
            }
            if (store) {
              const int k = left(col, 4);
              put64(out + (int64_t)col * 4, g32, wide, k);
              put64(out + (int64_t)col * 4 + 64, g32 + 16, wide, k - 4);
              put64(out + ((int64_t)P.N + col) * 4, u32, wide, k);
              put64(out + ((int64_t)P.N + col) * 4 + 64, u32 + 16, wide, k - 4);
              put64(act + (int64_t)col * 2, ap, wide, left(col, 2));
            }
          }
        } else if (some && KIND == kKDownGrad) {
          const int n0 = n * 256;
#pragma unroll 1
          for (int c = part * kCols; c < (part + 1) * kCols; c += 32) {
            const int col = n0 + c;
            if (col >= P.N) break;
            __syncwarp();
            uint32_t dv[32], dg[16], du[16], ap[16];
            tmem_ld32(tb + c, dv);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x[2], y[2], z[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int j = 2 * i + k;
                const float d = __uint_as_float(dv[j]), g = __uint_as_float(gq[j / 8][j % 8]);
                const float u = __uint_as_float(uq[j / 8][j % 8]), s = sigmoid(g);
                x[k] = d * u * s * (1.f + g * (1.f - s));
                y[k] = d * g * s;
                z[k] = g * s * u;
              }
              dg[i] = slot ? pack_bf16(x[0], x[1]) : 0u;
              du[i] = slot ? pack_bf16(y[0], y[1]) : 0u;
              ap[i] = slot ? pack_bf16(z[0], z[1]) : 0u;
            }
            if (c + 32 < (part + 1) * kCols) ask(col + 32);  // on their way during what follows
            if (store) {
              const int k = left(col, 2);
              put64(out + (int64_t)col * 2, dg, wide, k);
              put64(out + ((int64_t)P.N + col) * 2, du, wide, k);
              put64(act + (int64_t)col * 2, ap, wide, k);
            }
          }
        } else if (LY::staged && some) {
          // bf16 dW of short reductions: whole 128-byte lines through the TMA, as fp32 ones
          constexpr int W = 64;
          uint8_t* const t = smem + LY::out + (size_t)(warp - 2) * OUT_BYTES;
          const int n0 = n * 256;
#pragma unroll 1
          for (int c = part * kCols; c < (part + 1) * kCols; c += W) {
            const int col = n0 + c;
            if (col >= P.N) break;
            // the tile's last store has been read
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int x = 0; x < W; x += 32) {
              uint32_t v[32];
              __syncwarp();  // the aligned load below: the lanes part where some add old values
              if (computed) {
                tmem_ld32(tb + c + x, v);
                tmem_ld_wait();
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0;
              }
              if (P.accumulate && store) add_old(v, out + (int64_t)(col + x) * 2, wide, left(col + x, 2));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t p4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  p4[j] = pack_bf16(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1]));
                *piece(t, lane, x / 8 + i) = make_uint4(p4[0], p4[1], p4[2], p4[3]);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              store_3d(&TM.o, t, col, m, it.e);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          }
        } else if (some) {  // down, up_grad, bf16 dW of long reductions
          const int n0 = n * 256;
#pragma unroll 1
          for (int c = part * kCols; c < (part + 1) * kCols; c += 32) {
            const int col = n0 + c;
            if (col >= P.N) break;
            __syncwarp();
            uint32_t v[32];
            if (computed) {
              tmem_ld32(tb + c, v);
              tmem_ld_wait();
            }
            if (!slot) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0;
            }
            if (store) {
              const int k = left(col, 2);
              if (R::weight && P.accumulate) add_old(v, out + (int64_t)col * 2, wide, k);
              uint32_t pr[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                pr[i] = pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
              put64(out + (int64_t)col * 2, pr, wide, k);
            }
          }
        }
        if (computed) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            arrive_relaxed(&tempty[a], 0);
          }
          acc_phase ^= 1u << a;
          if (NH == 1) acc ^= 1;
        }
      }
    }
    if (LY::staged) {
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      __syncwarp();
    }
  }

  __syncthreads();
  if (*abort_flag) {  // let copies already in flight land before shared memory is released
    const uint64_t t0 = gtimer();
    while (gtimer() - t0 < 200000ull) {
    }
    __syncwarp();  // the clock lets lanes go one by one; what follows takes whole warps
  }
  cluster_sync();  // no remote arrival still targets this CTA; both CTAs are done with TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem_base, kTmemCols);
  }
}

template <int KIND, int NH>
static moe_status_t launch(const Maps& tm, Params P, int64_t max_rows_items, int resident_only,
                           int* resident_out, cudaStream_t s) {
  auto kern = expert_pair_kernel<KIND, NH>;
  constexpr size_t smem = Layout<KIND, NH>::bytes;
  constexpr int threads = Layout<KIND, NH>::kThreads;
  // persistent grid: as many CTA pairs as can be resident at once
  static thread_local int configured_dev = -1, resident = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_dev != dev) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms() / 2));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, (void*)kern, &cfg) != cudaSuccess ||
        clusters < 1) {
      cudaGetLastError();
      clusters = num_sms() / 2;
    }
    resident = std::min(clusters, num_sms() / 2);
    configured_dev = dev;
  }
  if (resident_only) {
    *resident_out = resident;
    return MOE_OK;
  }
  P.n_items = ceil_div(P.n_tiles, NH);
  const int64_t items = max_rows_items * P.n_items;
  const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(resident, items));
  return launch_k(kern, dim3(2 * pairs), dim3(threads), smem, s, tm, P);
}

// Wide items (NH = 2) take over from this reduction length on (average rows an expert for the weight
// gradients); below it the epilogue that they leave uncovered costs more than they save. Measured at
// 8 to 64 experts of 512 to 4096 rows, narrow against wide, us: up 2048 long 419 and 460, 4096 1326
// and 1290, 8192 1530 and 1392; down 1024 197 and 211, 2048 757 and 720, 14336 687 and 648; up_grad 2048
// 380 and 361, 4096 390 and 348; bf16 weights over 512 rows 247 and 271, 1024 1381 and 1396, 2048
// 1510 and 1412. Down_grad, whose epilogue reads the most, lost at every length (8192: 889 against 874 at best,
// 4096 801 and 935): it has no wide form, nor have fp32 weights, whose sums fill the registers.
template <int KIND>
constexpr int kWideFrom = KIND == kKUp         ? 4096
                          : KIND == kKDown     ? 2048
                          : KIND == kKUpGrad   ? 2048
                          : KIND == kKWeight16 ? 1536
                                               : 0;
// And from this many wide items a resident CTA pair on: with fewer, the last round leaves too many
// pairs without work.
constexpr int kWideRounds = 3;

// row_items: row tiles that are sure to have work (how they fall on the experts is known on the device
// only); max_row_items: the most there can be.
template <int KIND>
static moe_status_t launch_either(const Maps& tm, const Params& P, int reduction, int64_t row_items,
                                  int64_t max_row_items, cudaStream_t s) {
  if (max_row_items * P.n_tiles > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  if constexpr (kWideFrom<KIND> > 0) {
    int resident = 0;
    const moe_status_t st = launch<KIND, 2>(tm, P, 0, 1, &resident, s);
    if (st != MOE_OK) return st;
    if (reduction >= kWideFrom<KIND> &&
        row_items * ceil_div(P.n_tiles, 2) >= (int64_t)kWideRounds * resident)
      return launch<KIND, 2>(tm, P, max_row_items, 0, nullptr, s);
  }
  return launch<KIND, 1>(tm, P, max_row_items, 0, nullptr, s);
}

}  // namespace etc

using namespace etc;

int experts_tc_status_read(int reset) {
  int v = 0;
  cudaMemcpyFromSymbol(&v, etc::g_status, sizeof(int));
  if (reset) {
    int z = 0;
    cudaMemcpyToSymbol(etc::g_status, &z, sizeof(int));
  }
  return v;
}

moe_status_t launch_expert_product_tc(ExpertProduct kind, const moe_experts_t& c, const void* a,
                                      const void* w, const float* h13, const int32_t* counts,
                                      void* out, void* act, cudaStream_t s) {
  const uint64_t H = c.H, I = c.I, E = c.E, rows = c.rows;
  Maps tm;
  Params P{};
  P.counts = counts;
  P.h13 = h13;
  P.out = out;
  P.act = act;
  P.E = c.E;
  P.rows = c.rows;
  const bool up = kind == kUp, dgrad = kind == kDownGrad;
  P.N = up || dgrad ? c.I : c.H;
  P.K = up || dgrad ? c.H : kind == kDown ? c.I : 2 * c.I;
  P.n_tiles = ceil_div(P.N, up ? 128 : 256);
  P.out_bytes = up ? c.I * 8 : dgrad ? c.I * 4 : c.H * 2;
  P.act_bytes = up || dgrad ? c.I * 2 : 0;
  bool ok = true;
  {
    const uint64_t K = P.K;
    uint64_t d[2] = {K, rows}, st[1] = {K};
    uint32_t box[2] = {BK, 128};
    ok &= make_map(&tm.a, a, 2, d, st, box, false);
  }
  if (up) {
    uint64_t d[3] = {H, I, E}, st[2] = {H, 2 * I * H};
    uint32_t box[3] = {BK, 128, 1};
    ok &= make_map(&tm.b0, w, 3, d, st, box, true);
    ok &= make_map(&tm.b1, (const __nv_bfloat16*)w + I * H, 3, d, st, box, true);
  } else if (kind == kDown) {
    uint64_t d[3] = {I, H, E}, st[2] = {I, H * I};
    uint32_t box[3] = {BK, 128, 1};
    ok &= make_map(&tm.b0, w, 3, d, st, box, true);
  } else {
    // the weight with its columns contiguous along N: [K, N] of one expert
    const uint64_t N = P.N, K = P.K;
    uint64_t d[3] = {N, K, E}, st[2] = {N, K * N};
    uint32_t box[3] = {64, BK, 1};
    ok &= make_map(&tm.b0, w, 3, d, st, box, true);
  }
  if (!ok) return MOE_ERR_CUDA;
  P.wide = (((uintptr_t)out | (uintptr_t)act | (uintptr_t)h13) & 31u) == 0 && P.N % 16 == 0;
  const int64_t least = ceil_div(c.rows, 256), most = (int64_t)c.rows / 256 + c.E;
  switch (kind) {
    case kUp: return launch_either<kKUp>(tm, P, P.K, least, most, s);
    case kDown: return launch_either<kKDown>(tm, P, P.K, least, most, s);
    case kDownGrad: return launch_either<kKDownGrad>(tm, P, P.K, least, most, s);
    default: return launch_either<kKUpGrad>(tm, P, P.K, least, most, s);
  }
}

moe_status_t launch_weight_grad_tc(int rows, int E, int M, int N, moe_dtype_t out_dt,
                                   int accumulate, const void* dy, const void* a,
                                   const int32_t* counts, void* dW, cudaStream_t s) {
  const uint64_t m = M, n = N, r = rows;
  Maps tm;
  Params P{};
  P.counts = counts;
  P.out = dW;
  P.E = E;
  P.rows = rows;
  P.M = M;
  P.N = N;
  P.m_tiles = ceil_div(M, 256);
  P.n_tiles = ceil_div(N, 256);
  P.accumulate = accumulate;
  const bool f32 = out_dt == MOE_F32;
  P.out_bytes = N * (f32 ? 4 : 2);
  uint32_t box[2] = {64, BK};
  uint64_t da[2] = {m, r}, sa[1] = {m}, db[2] = {n, r}, sb[1] = {n};
  bool ok = make_map(&tm.a, dy, 2, da, sa, box, false) && make_map(&tm.b0, a, 2, db, sb, box, false);
  box[1] = 16;
  ok = ok && make_map(&tm.a16, dy, 2, da, sa, box, false) && make_map(&tm.b16, a, 2, db, sb, box, false);
  {
    auto fn = encode_fn();
    cuuint64_t d[3] = {n, m, (uint64_t)E}, st[2] = {n * (f32 ? 4 : 2), m * n * (f32 ? 4 : 2)};
    cuuint32_t obox[3] = {f32 ? 32u : 64u, 32u, 1u}, one[3] = {1, 1, 1};
    ok = ok && fn && fn(&tm.o, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        dW, d, st, obox, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  if (!ok) return MOE_ERR_CUDA;
  P.wide = ((uintptr_t)dW & 31u) == 0 && P.out_bytes % 32 == 0;
  const int64_t items = (int64_t)E * P.m_tiles;
  return f32 ? launch_either<kKWeight32>(tm, P, rows / E, items, items, s)
             : launch_either<kKWeight16>(tm, P, rows / E, items, items, s);
}

}  // namespace moe
