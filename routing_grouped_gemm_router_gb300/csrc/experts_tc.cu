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
// makes the weight gradient's reduction exact without masks, and lets every 16-row box of an
// output belong to one expert, so results leave through the TMA: registers -> a swizzled 4 KB
// tile a warp -> cp.async.bulk.tensor store, full 128-byte lines, ragged edges clipped by the map.
//
// Roles in each CTA of a pair: warp 0 issues the TMA loads into a ring of 32 KB stages, warp 1 of
// the leader issues the MMAs, warps 2-5 are the epilogue over double-buffered accumulators. Work
// items are (expert, 256-row or 256-column tile, 256-column tile), weight panels outermost within
// an expert, so that pairs running together share them in L2; persistent CTA pairs take them in
// turn. All waits are bounded (status kStatusTimeout, no trap).
#include "tc_ptx.cuh"
#include "train.cuh"

namespace moe {
namespace etc {

using namespace ptx;

__device__ int g_status;

enum Kind { kKUp = 0, kKDown = 1, kKDownGrad = 2, kKUpGrad = 3, kKWeight32 = 4, kKWeight16 = 5 };

constexpr int kStages = 5;
constexpr int kAccs = 2;
constexpr int kTmemCols = 512;
constexpr int kThreads = 192;
constexpr int A_BYTES = 128 * 128;
constexpr int B_BYTES = 128 * 128;
constexpr int CHUNK = 64 * 128;    // one 64-column box of an M/N-major operand: 64 K rows x 128 B
constexpr int OUT_BYTES = 32 * 128;  // one staged output tile of a warp
constexpr int kOutBufs = 3;        // a warp's tiles: written, being read by the TMA, free

template <int KIND>
struct Traits {
  static constexpr bool weight = KIND >= kKWeight32;
  static constexpr bool a_mn = weight;  // operand contiguous along M rather than K
  static constexpr bool b_mn = KIND >= kKDownGrad;
  // columns of the result an item covers
  static constexpr int cols = KIND == kKUp ? 128 : 256;
  static constexpr uint32_t idesc =
      idesc_bf16(256, 256) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
};

struct Layout {
  static constexpr size_t a = 0;
  static constexpr size_t b = a + (size_t)kStages * A_BYTES;
  static constexpr size_t out = b + (size_t)kStages * B_BYTES;
  static constexpr size_t bars = out + (size_t)4 * kOutBufs * OUT_BYTES;
  static constexpr size_t misc = bars + (2 * kStages + 5) * 8;
  static constexpr size_t start = misc + 16;
  static constexpr size_t cnt = start + (kMaxExperts + 1) * 4;
  static constexpr size_t pre = cnt + kMaxExperts * 4;
  static constexpr size_t end = pre + (kMaxExperts + 1) * 4;
  static constexpr size_t bytes = 1024 + end;
};
static_assert(Layout::bytes <= 232448, "shared memory");

struct Params {
  const int32_t* counts;
  const float* h13;  // down_grad: the pre-activations [rows, 2I]
  void* out;         // zeroed tail rows: rows of out_bytes each
  void* act;         // and of act_bytes each (up, down_grad)
  int E, rows;
  int M;             // weight: rows of dW[e]
  int N;             // columns of the result (up: I)
  int K;             // reduction (rows kinds)
  int m_tiles, n_tiles;
  int accumulate;
  int out_bytes, act_bytes;
};

struct Maps {
  CUtensorMap a, b0, b1, o0, o1, o2;
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

__device__ __forceinline__ void store_2d(const CUtensorMap* tm, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   (uint64_t)tm),
               "r"(c0), "r"(c1), "r"(su32(src))
               : "memory");
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
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void store_wait_read() {  // all but the N latest groups have been read
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// The 16-byte piece c of row r of a staged tile (128-byte swizzle, as the output map has it).
__device__ __forceinline__ uint4* piece(uint8_t* tile, int r, int c) {
  return reinterpret_cast<uint4*>(tile + r * 128 + ((c ^ (r & 7)) << 4));
}
// Thirty-two fp32 values of row r: a whole row of an fp32 tile.
__device__ __forceinline__ void stage_f32(uint8_t* tile, int r, const uint32_t (&v)[32], bool keep) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *piece(tile, r, c) = keep ? make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3])
                              : make_uint4(0, 0, 0, 0);
}
// Thirty-two values as bf16: the `half`-th 64 bytes of a row of a bf16 tile.
__device__ __forceinline__ void stage_bf16(uint8_t* tile, int r, int half, const float (&v)[32],
                                           bool keep) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *piece(tile, r, half * 4 + c) =
        keep ? make_uint4(pack_bf16(v[8 * c], v[8 * c + 1]), pack_bf16(v[8 * c + 2], v[8 * c + 3]),
                          pack_bf16(v[8 * c + 4], v[8 * c + 5]), pack_bf16(v[8 * c + 6], v[8 * c + 7]))
             : make_uint4(0, 0, 0, 0);
}

struct Item {
  int e, n;        // expert, column tile
  int m0;          // first row of the tile (weight: first row of dW[e])
  int row0, cnt;   // the expert's rows
  int num_kb;
  bool live1;      // the peer's half of the tile holds rows
};

template <int KIND>
__device__ __forceinline__ Item item_of(int w, const Params& P, const int* start, const int* cnt,
                                        const int* pre) {
  Item it;
  if (Traits<KIND>::weight) {
    const int per = P.m_tiles * P.n_tiles;
    it.e = w / per;
    const int rest = w - it.e * per;
    it.n = rest % P.n_tiles;
    it.m0 = rest / P.n_tiles * 256;
    it.row0 = start[it.e];
    it.cnt = cnt[it.e];
    it.num_kb = (it.cnt + BK - 1) / BK;
    it.live1 = true;
  } else {
    int lo = 0, hi = P.E - 1;  // the last expert whose first item is at or before w
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * P.n_tiles <= w) lo = mid; else hi = mid - 1;
    }
    const int c = pre[lo + 1] - pre[lo];
    const int local = w - pre[lo] * P.n_tiles;
    it.e = lo;
    it.n = local / c;
    const int i = local - it.n * c;
    it.row0 = start[lo];
    it.cnt = cnt[lo];
    it.m0 = it.row0 + i * 256;
    it.num_kb = (P.K + BK - 1) / BK;
    it.live1 = i * 256 + 128 < it.cnt;
  }
  return it;
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expert_pair_kernel(const __grid_constant__ Maps TM, const Params P) {
  using R = Traits<KIND>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sA = smem + Layout::a;
  uint8_t* sB = smem + Layout::b;
  uint64_t* full = (uint64_t*)(smem + Layout::bars);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = (uint32_t*)(smem + Layout::misc);
  volatile int* abort_flag = (volatile int*)(smem + Layout::misc + 4);
  int* start = (int*)(smem + Layout::start);
  int* cnt = (int*)(smem + Layout::cnt);
  int* pre = (int*)(smem + Layout::pre);
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
      mbar_init(&tempty[b], 8);  // four epilogue warps of each CTA (the leader's is used)
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
    prefetch_tmap(&TM.a);
    prefetch_tmap(&TM.b0);
    prefetch_tmap(&TM.o0);
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
  const int total = R::weight ? P.E * P.m_tiles * P.n_tiles : pre[P.E] * P.n_tiles;
  const int pair = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int g = 0;
      bool ok = true;
      for (int w = pair; w < total && ok; w += num_pairs) {
        const Item it = item_of<KIND>(w, P, start, cnt, pre);
        for (int kb = 0; kb < it.num_kb; ++kb, ++g) {
          const int s = g % kStages;
          if (!wait_bounded(&empty[s], ((uint32_t)(g / kStages) & 1u) ^ 1u, abort_flag, status)) {
            ok = false;
            break;
          }
          const uint32_t fl = cluster_addr(&full[s], 0);
          if (leader)
            mbar_expect_tx(&full[s], 2u * (A_BYTES + B_BYTES) - (it.live1 ? 0u : (uint32_t)A_BYTES));
          uint8_t* a = sA + s * A_BYTES;
          uint8_t* b = sB + s * B_BYTES;
          if (R::weight) {
            const int y = it.row0 + kb * BK, m = it.m0 + (int)rank * 128, n = it.n * 256 + (int)rank * 128;
            tma_2d_pair(a, &TM.a, fl, m, y);
            tma_2d_pair(a + CHUNK, &TM.a, fl, m + 64, y);
            tma_2d_pair(b, &TM.b0, fl, n, y);
            tma_2d_pair(b + CHUNK, &TM.b0, fl, n + 64, y);
          } else {
            // the peer's rows of a half-filled tile are neither loaded nor stored
            if (leader || it.live1) tma_2d_pair(a, &TM.a, fl, kb * BK, it.m0 + (int)rank * 128);
            if (KIND == kKUp) {  // leader: gate rows, peer: the same up rows
              tma_3d_pair(b, rank ? &TM.b1 : &TM.b0, fl, kb * BK, it.n * 128, it.e);
            } else if (KIND == kKDown) {
              tma_3d_pair(b, &TM.b0, fl, kb * BK, it.n * 256 + (int)rank * 128, it.e);
            } else {
              const int n = it.n * 256 + (int)rank * 128;
              tma_3d_pair(b, &TM.b0, fl, n, kb * BK, it.e);
              tma_3d_pair(b + CHUNK, &TM.b0, fl, n + 64, kb * BK, it.e);
            }
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ leader: MMA issuer
    if (leader && lane == 0) {
      int g = 0, acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true, issued = false;
      for (int w = pair; w < total && ok; w += num_pairs) {
        const Item it = item_of<KIND>(w, P, start, cnt, pre);
        if (it.num_kb == 0) continue;
        if (!wait_bounded(&tempty[acc], acc_phase ^ 1u, abort_flag, status)) break;
        tc_fence_after();
        if (*abort_flag) break;
        const uint32_t d = tmem_base + (uint32_t)(acc * 256);
        const int K = R::weight ? it.cnt : P.K;
        for (int kb = 0; kb < it.num_kb; ++kb, ++g) {
          const int s = g % kStages;
          if (!wait_bounded(&full[s], (uint32_t)(g / kStages) & 1u, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = su32(sA + s * A_BYTES), b = su32(sB + s * B_BYTES);
          const int steps = min(BK / UMMA_K, (K - kb * BK + UMMA_K - 1) / UMMA_K);
#pragma unroll
          for (int kk = 0; kk < BK / UMMA_K; ++kk) {
            if (kk < steps)
              umma_bf16<2>(d, R::a_mn ? mn_desc(a + kk * 2048) : sw128_desc(a + kk * 32),
                           R::b_mn ? mn_desc(b + kk * 2048) : sw128_desc(b + kk * 32), R::idesc,
                           (kb | kk) != 0 ? 1u : 0u);
          }
          umma_commit_pair(&empty[s], 0x3);
          issued = true;
        }
        if (!ok) break;
        umma_commit_pair(&tfull[acc], 0x3);
        if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
      }
      if (issued) {  // every MMA of this thread finished before tensor memory is freed
        umma_commit<2>(drain);
        wait_bounded(drain, 0, abort_flag, status);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (4 warps)
    const int q = warp & 3;  // tensor-memory lanes q*32 .. q*32+31
    uint8_t* tiles = smem + Layout::out + (size_t)(warp - 2) * kOutBufs * OUT_BYTES;
    int buf = 0;
    if (!R::weight) {  // rows past the last run are zeroed while the first tile is computed
      const int t = (warp - 2) * 32 + lane;
      const uint4 z = make_uint4(0, 0, 0, 0);
      for (int p = start[P.E] + (int)blockIdx.x; p < P.rows; p += gridDim.x) {
        for (int v = t; v < P.out_bytes / 16; v += 128)
          ((uint4*)((uint8_t*)P.out + (int64_t)p * P.out_bytes))[v] = z;
        for (int v = t; v < P.act_bytes / 16; v += 128)
          ((uint4*)((uint8_t*)P.act + (int64_t)p * P.act_bytes))[v] = z;
      }
    }
    // the next staged tile, once the TMA has read what it held three stores ago
    auto next_tile = [&]() {
      if (lane == 0) store_wait_read<kOutBufs - 1>();
      __syncwarp();
      uint8_t* t = tiles + buf * OUT_BYTES;
      buf = buf + 1 == kOutBufs ? 0 : buf + 1;
      return t;
    };
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int w = pair; w < total; w += num_pairs) {
      const Item it = item_of<KIND>(w, P, start, cnt, pre);
      if (R::weight && it.num_kb == 0 && P.accumulate) continue;
      const bool computed = it.num_kb != 0;
      if (computed) {
        int ok = 1;
        if (lane == 0) ok = wait_bounded(&tfull[acc], acc_phase, abort_flag, status);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t tb = tmem_base + (uint32_t)(acc * 256) + ((uint32_t)(q * 32) << 16);
      const int m = it.m0 + (int)rank * 128 + q * 32;  // first row of this warp's 32
      auto load = [&](uint32_t (&v)[32], int col) {
        tmem_ld32(tb + col, v);
        tmem_ld_wait();
      };
      if (R::weight) {
        // dW[e][m .. m+31][...]: whole 32-row boxes, edges clipped by the map
        constexpr int W = KIND == kKWeight32 ? 32 : 64;
        const int n0 = it.n * 256;
#pragma unroll 1
        for (int c = 0; c < 256; c += W) {
          if (n0 + c >= P.N || m >= P.M) break;
          uint8_t* t = next_tile();
          if (KIND == kKWeight32) {
            uint32_t v[32];
            if (computed) load(v, c);
            stage_f32(t, lane, v, computed);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[32];
              float f[32];
              if (computed) load(v, c + 32 * h);
#pragma unroll
              for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
              if (P.accumulate && m + lane < P.M) {  // one rounding of the sum
                const __nv_bfloat16* old = (const __nv_bfloat16*)P.out +
                                           ((int64_t)it.e * P.M + m + lane) * P.N + n0 + c + 32 * h;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (n0 + c + 32 * h + 8 * i < P.N) {
                    float o[8];
                    Vec<__nv_bfloat16>::unpack(((const uint4*)old)[i], o);
#pragma unroll
                    for (int x = 0; x < 8; ++x) f[8 * i + x] += o[x];
                  }
              }
              stage_bf16(t, lane, h, f, computed);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (KIND == kKWeight32 && P.accumulate) add_3d(&TM.o0, t, n0 + c, m, it.e);
            else store_3d(&TM.o0, t, n0 + c, m, it.e);
            store_commit();
          }
        }
      } else {
        // 16-row boxes up to the run's padded end; rows past cnt are stored as zeros
        const int end = min(it.row0 + (it.cnt + kRowBlock - 1) / kRowBlock * kRowBlock, P.rows);
        const bool slot = m + lane < it.row0 + it.cnt;
        // one group a tile, empty where nothing is stored: next_tile counts groups
        auto put = [&](const CUtensorMap* tm, uint8_t* t, int col) {
          if (lane == 0) {
            if (col < P.N && m < end) store_2d(tm, t, col, m);
            if (col < P.N && m + 16 < end) store_2d(tm, t + 16 * 128, col, m + 16);
            store_commit();
          }
        };
        if (KIND == kKUp) {
          const int n0 = it.n * 128;
#pragma unroll 1
          for (int c = 0; c < 128 && m < end; c += 64) {
            if (n0 + c >= P.N) break;
            uint32_t ap[32];  // the 64 activations as bf16 pairs
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t gv[32], uv[32];
              tmem_ld32(tb + c + 32 * h, gv);
              tmem_ld32(tb + 128 + c + 32 * h, uv);
              tmem_ld_wait();
              uint8_t* tg = next_tile();
              stage_f32(tg, lane, gv, slot);
              fence_proxy_async_smem();
              __syncwarp();
              put(&TM.o0, tg, n0 + c + 32 * h);
              uint8_t* tu = next_tile();
              stage_f32(tu, lane, uv, slot);
              fence_proxy_async_smem();
              __syncwarp();
              put(&TM.o1, tu, n0 + c + 32 * h);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float a2[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const float g = __uint_as_float(gv[2 * i + x]);
                  a2[x] = g * (1.f / (1.f + expf(-g))) * __uint_as_float(uv[2 * i + x]);
                }
                ap[16 * h + i] = slot ? pack_bf16(a2[0], a2[1]) : 0u;
              }
            }
            uint8_t* ta = next_tile();
#pragma unroll
            for (int p = 0; p < 8; ++p)
              *piece(ta, lane, p) = make_uint4(ap[4 * p], ap[4 * p + 1], ap[4 * p + 2], ap[4 * p + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            put(&TM.o2, ta, n0 + c);
          }
        } else if (KIND == kKDownGrad) {
          const int n0 = it.n * 256;
          const float* hrow = P.h13 + (int64_t)(m + lane) * 2 * P.N;
#pragma unroll 1
          for (int c = 0; c < 256 && m < end; c += 64) {
            if (n0 + c >= P.N) break;
            uint8_t *tg = next_tile(), *tu = next_tile(), *ta = next_tile();
            if (lane == 0) store_wait_read<0>();  // all three are written at once
            __syncwarp();
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              const int col = n0 + c + 32 * h;
              float gv[32], uv[32];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                if (slot && col + 4 * i < P.N) {
                  a = __ldg((const float4*)(hrow + col) + i);
                  b = __ldg((const float4*)(hrow + P.N + col) + i);
                }
                gv[4 * i] = a.x; gv[4 * i + 1] = a.y; gv[4 * i + 2] = a.z; gv[4 * i + 3] = a.w;
                uv[4 * i] = b.x; uv[4 * i + 1] = b.y; uv[4 * i + 2] = b.z; uv[4 * i + 3] = b.w;
              }
              uint32_t dv[32];
              load(dv, c + 32 * h);
              float av[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float d = __uint_as_float(dv[i]), g = gv[i], u = uv[i];
                const float s = 1.f / (1.f + expf(-g));
                av[i] = g * s * u;
                gv[i] = d * u * s * (1.f + g * (1.f - s));
                uv[i] = d * g * s;
              }
              stage_bf16(tg, lane, h, gv, slot);
              stage_bf16(tu, lane, h, uv, slot);
              stage_bf16(ta, lane, h, av, slot);
            }
            fence_proxy_async_smem();
            __syncwarp();
            put(&TM.o0, tg, n0 + c);
            put(&TM.o1, tu, n0 + c);
            put(&TM.o2, ta, n0 + c);
          }
        } else {
          const int n0 = it.n * 256;
#pragma unroll 1
          for (int c = 0; c < 256 && m < end; c += 64) {
            if (n0 + c >= P.N) break;
            uint8_t* t = next_tile();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[32];
              float f[32];
              load(v, c + 32 * h);
#pragma unroll
              for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
              stage_bf16(t, lane, h, f, slot);
            }
            fence_proxy_async_smem();
            __syncwarp();
            put(&TM.o0, t, n0 + c);
          }
        }
      }
      if (computed) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&tempty[acc]);
          else mbar_arrive_cta(&tempty[acc], 0);
        }
        if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  __syncthreads();
  if (*abort_flag) {  // let copies already in flight land before shared memory is released
    const uint64_t t0 = gtimer();
    while (gtimer() - t0 < 200000ull) {
    }
  }
  cluster_sync();  // no remote arrival still targets this CTA; both CTAs are done with TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem_base, kTmemCols);
  }
}

// Output map: boxes of 128-byte rows, 128-byte swizzle.
static bool make_out_map(CUtensorMap* m, void* base, bool f32, int rank, const uint64_t* dims,
                         const uint64_t* strides_elems, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t gdim[3], gstr[2];
  cuuint32_t bdim[3] = {f32 ? 32u : 64u, box_rows, 1u}, estr[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) gdim[i] = dims[i];
  for (int i = 0; i + 1 < rank; ++i) gstr[i] = strides_elems[i] * (f32 ? 4 : 2);
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base,
            gdim, gstr, bdim, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND>
static moe_status_t launch(const Maps& tm, const Params& P, int64_t max_items, cudaStream_t s) {
  auto kern = expert_pair_kernel<KIND>;
  constexpr size_t smem = Layout::bytes;
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
    cfg.blockDim = dim3(kThreads);
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
  const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(resident, max_items));
  return launch_k(kern, dim3(2 * pairs), dim3(kThreads), smem, s, tm, P);
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
    uint64_t od[2] = {I, rows}, os[1] = {2 * I}, as[1] = {I};
    ok &= make_out_map(&tm.o0, out, true, 2, od, os, 16);
    ok &= make_out_map(&tm.o1, (float*)out + I, true, 2, od, os, 16);
    ok &= make_out_map(&tm.o2, act, false, 2, od, as, 16);
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
  if (dgrad) {
    uint64_t od[2] = {I, rows}, os[1] = {2 * I}, as[1] = {I};
    ok &= make_out_map(&tm.o0, out, false, 2, od, os, 16);
    ok &= make_out_map(&tm.o1, (__nv_bfloat16*)out + I, false, 2, od, os, 16);
    ok &= make_out_map(&tm.o2, act, false, 2, od, as, 16);
  } else if (!up) {
    uint64_t od[2] = {H, rows}, os[1] = {H};
    ok &= make_out_map(&tm.o0, out, false, 2, od, os, 16);
  }
  if (!ok) return MOE_ERR_CUDA;
  const int64_t items = ((int64_t)c.rows / 256 + c.E) * P.n_tiles;
  if (items > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  switch (kind) {
    case kUp: return launch<kKUp>(tm, P, items, s);
    case kDown: return launch<kKDown>(tm, P, items, s);
    case kDownGrad: return launch<kKDownGrad>(tm, P, items, s);
    default: return launch<kKUpGrad>(tm, P, items, s);
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
  uint32_t box[2] = {64, BK};
  uint64_t da[2] = {m, r}, sa[1] = {m}, db[2] = {n, r}, sb[1] = {n};
  uint64_t dw[3] = {n, m, (uint64_t)E}, sw[2] = {n, m * n};
  if (!make_map(&tm.a, dy, 2, da, sa, box, false) || !make_map(&tm.b0, a, 2, db, sb, box, false) ||
      !make_out_map(&tm.o0, dW, f32, 3, dw, sw, 32))
    return MOE_ERR_CUDA;
  const int64_t items = (int64_t)E * P.m_tiles * P.n_tiles;
  if (items > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  return f32 ? launch<kKWeight32>(tm, P, items, s) : launch<kKWeight16>(tm, P, items, s);
}

}  // namespace moe
