// dispatch.cu — token rows sorted by expert and back, with the router weights, and the
// gradients of both (moe_permute, moe_unpermute and their backward calls).
//
// With pos[t, j] the row of slot j of token t in the expert-sorted buffer:
//   permute             xs[pos[t, j]] = x[t]
//   its gradient        dx[t] = sum_j dxs[pos[t, j]]
//   unpermute           out[t] = sum_j w[t, j] ys[pos[t, j]]
//   its gradients       dys[pos[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], ys[pos[t, j]]>
// All four move rows and do next to no arithmetic, so HBM bounds them: every row is read and
// written once, in 16-byte pieces. Sums over slots and over a row are fp32, in a fixed order.
#include "train.cuh"

namespace moe {
namespace dispatch {

// ------------------------------------------------------------------- permute
// One warp a buffer row: the sorted table gives the slot, the slot its token. Rows of no slot are
// written as zeros, so that the expert products may run over whole 16-row steps. Written rows are
// marked to leave L2 first, for the token rows that are read k times to stay.
__global__ void __launch_bounds__(256) permute_kernel(const uint4* __restrict__ x,
                                                      const int32_t* __restrict__ ids,
                                                      const int32_t* __restrict__ sid, int n,
                                                      int k, int E, int rows, int vec,
                                                      uint4* __restrict__ xs,
                                                      int32_t* __restrict__ pos) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  // slots without an expert never appear in the table: their position is written here
  for (int r = blockIdx.x * blockDim.x + threadIdx.x; r < n; r += gridDim.x * blockDim.x) {
    const int e = ids[r];
    if (e < 0 || e >= E) pos[r] = -1;
  }
  const int warps = gridDim.x * (blockDim.x >> 5);
  for (int p = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); p < rows; p += warps) {
    const int r = sid[p];
    uint4* dst = xs + (int64_t)p * vec;
    if (r < 0 || r >= n) {
      const uint4 z = make_uint4(0, 0, 0, 0);
      for (int v = lane; v < vec; v += 32) dst[v] = z;
      continue;
    }
    if (lane == 0) pos[r] = p;
    const uint4* src = x + (int64_t)(r / k) * vec;
    int v = lane;
    for (; v + 96 < vec; v += 128) {
      const uint4 a = src[v], b = src[v + 32], c = src[v + 64], d = src[v + 96];
      __stcs(dst + (v), a);
      __stcs(dst + (v + 32), b);
      __stcs(dst + (v + 64), c);
      __stcs(dst + (v + 96), d);
    }
    for (; v < vec; v += 32) __stcs(dst + v, src[v]);
  }
}

// Where the copies outgrow L2, token rows would come from HBM several times that way (199 MB read for
// 58 MB of tokens: 114 us for 4096 x 7168 with 8 slots each). So positions are written first, by a
// kernel of their own, and then a thread reads a 16-byte piece of a token once and writes it to the
// token's k rows: 89 us, 5.9 TB/s written. The first blocks write the rows of no slot. Row-major against
// token-major over 64 experts, us, 2048 and 7168 channels: xs of 64 MB 13 to 16 and 12 to 22, 128 MB 27 to 39
// and 25 to 33, 256 MB 56 to 79 and 49 to 62, 512 MB 125 to 165 and 94 to 121 (2, 4 and 8 slots a token). With
// one slot nothing is read twice: 43 and 44 us at 128 MB, 167 and 169 at 512.
constexpr size_t kTokenMajorFrom = (size_t)1 << 27;  // bytes of xs, for two slots a token or more
constexpr int kZeroRows = 64;                        // table entries a zeroing block looks at

__global__ void __launch_bounds__(256) positions_kernel(const int32_t* __restrict__ ids,
                                                        const int32_t* __restrict__ sid, int n,
                                                        int E, int rows, int32_t* __restrict__ pos) {
  pdl_wait();
  pdl_trigger();
  const int first = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
  for (int r = first; r < n; r += step) {
    const int e = ids[r];
    if (e < 0 || e >= E) pos[r] = -1;
  }
  for (int p = first; p < rows; p += step) {
    const int r = sid[p];
    if (r >= 0 && r < n) pos[r] = p;
  }
}

// Zeros into the rows of no slot among table entries block * kZeroRows ..., a warp a row.
__device__ __forceinline__ void zero_rows(int block, const int32_t* __restrict__ sid, int n, int rows,
                                          int vec, uint4* __restrict__ xs) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int p0 = block * kZeroRows;
  for (int p = p0 + (threadIdx.x >> 5); p < min(p0 + kZeroRows, rows); p += warps) {
    const int r = sid[p];
    if (r >= 0 && r < n) continue;
    for (int v = lane; v < vec; v += 32) __stcs(xs + (int64_t)p * vec + v, make_uint4(0, 0, 0, 0));
  }
}

__global__ void __launch_bounds__(256) permute_tokens_kernel(
    const uint4* __restrict__ x, const int32_t* __restrict__ sid, const int32_t* __restrict__ pos,
    int Tn, int k, int rows, int vec, int parts, uint4* __restrict__ xs) {
  pdl_wait();
  pdl_trigger();
  const int zeroing = (rows + kZeroRows - 1) / kZeroRows;
  if ((int)blockIdx.x < zeroing) {
    zero_rows(blockIdx.x, sid, Tn * k, rows, vec, xs);
    return;
  }
  const int b = blockIdx.x - zeroing;
  const int64_t t = b / parts;
  const int v = b % parts * blockDim.x + threadIdx.x;
  if (v >= vec) return;
  const uint4 q = __ldcs(x + t * vec + v);
  for (int j = 0; j < k; ++j) {
    const int p = __ldg(pos + t * k + j);
    if (p >= 0 && p < rows) __stcs(xs + (int64_t)p * vec + v, q);
  }
}

// ------------------------------------------------- sums over a token's slots
// One thread a 16-byte piece of a token's row; the slots' pieces are loaded four at a time
// before any is added, so four rows are in flight a thread.
template <typename T, bool WEIGHTED>
__global__ void __launch_bounds__(256) slot_sum_kernel(const uint4* __restrict__ ys,
                                                       const int32_t* __restrict__ pos,
                                                       const float* __restrict__ w, int k,
                                                       int rows, int vec, int parts,
                                                       uint4* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x / parts;
  const int v = (int)(blockIdx.x % parts) * blockDim.x + threadIdx.x;
  if (v >= vec) return;
  constexpr int W = 16 / sizeof(T);
  float acc[W];
#pragma unroll
  for (int i = 0; i < W; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < k; j0 += 4) {
    uint4 q[4];
    float wj[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = j0 + j < k ? __ldg(pos + t * k + j0 + j) : -1;
      const bool live = p >= 0 && p < rows;
      q[j] = live ? __ldcs(ys + (int64_t)p * vec + v) : make_uint4(0, 0, 0, 0);
      wj[j] = WEIGHTED && live ? __ldg(w + t * k + j0 + j) : (live ? 1.f : 0.f);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[W];
      Vec<T>::unpack(q[j], f);
#pragma unroll
      for (int i = 0; i < W; ++i) acc[i] = WEIGHTED ? fmaf(wj[j], f[i], acc[i]) : acc[i] + f[i];
    }
  }
  out[t * vec + v] = Vec<T>::pack(acc);
}

// ------------------------------------------------- gradients of the weighted sum
// One block a token. Its slots are taken four at a time: a thread loads its 16-byte piece
// of dout and of the four ys rows before it uses any, so that four rows are in flight; the dot
// products of all slots meet in shared memory once, at the end. (dout comes from L2 again for
// the next four.) The first blocks write zeros into rows of no slot.
constexpr int kUbThreads = 256;
constexpr int kBatch = 4;

template <typename T>
__global__ void __launch_bounds__(kUbThreads) unpermute_backward_kernel(
    const uint4* __restrict__ dout, const uint4* __restrict__ ys, const int32_t* __restrict__ sid,
    const int32_t* __restrict__ pos, const float* __restrict__ w, int Tn, int k, int rows,
    int vec, uint4* __restrict__ dys, float* __restrict__ dw) {
  pdl_wait();
  pdl_trigger();
  constexpr int W = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int zeroing = (rows + kZeroRows - 1) / kZeroRows;
  if ((int)blockIdx.x < zeroing) {
    zero_rows(blockIdx.x, sid, Tn * k, rows, vec, dys);
    return;
  }
  __shared__ float dots[32][kUbThreads / 32];
  const int64_t t = (int)blockIdx.x - zeroing;
  const uint4* drow = dout + t * vec;
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    const uint4* yrow[kBatch];
    uint4* orow[kBatch];
    float wj[kBatch], dot[kBatch];
    bool live[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int p = j0 + j < k ? __ldg(pos + t * k + j0 + j) : -1;
      live[j] = p >= 0 && p < rows;
      wj[j] = live[j] ? __ldg(w + t * k + j0 + j) : 0.f;
      const int64_t at = (int64_t)(live[j] ? p : 0) * vec;
      yrow[j] = ys + at;
      orow[j] = dys + at;
      dot[j] = 0.f;
    }
    for (int v = threadIdx.x; v < vec; v += blockDim.x) {
      const uint4 dq = drow[v];
      uint4 yq[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (live[j]) yq[j] = __ldcs(yrow[j] + v);
      float d[W];
      Vec<T>::unpack(dq, d);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (!live[j]) continue;
        float y[W];
        Vec<T>::unpack(yq[j], y);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          dot[j] = fmaf(d[i], y[i], dot[j]);
          y[i] = d[i] * wj[j];
        }
        __stcs(orow[j] + v, Vec<T>::pack(y));
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float s = warp_total(dot[j]);
      if (lane == 0 && j0 + j < k) dots[j0 + j][warp] = s;
    }
  }
  __syncthreads();
  if (threadIdx.x < k) {
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += dots[threadIdx.x][i];
    dw[t * k + threadIdx.x] = s;
  }
}

}  // namespace dispatch

using namespace dispatch;

moe_status_t launch_permute(const void* x, const int32_t* ids, const int32_t* sid, int T, int k,
                            int E, int H, moe_dtype_t dt, int rows, void* xs, int32_t* pos,
                            cudaStream_t s) {
  const int vec = H * (int)dtype_size(dt) / 16;
  const int threads = vec >= 256 ? 256 : std::max(32, ceil_div(vec, 32) * 32);
  const int parts = ceil_div(vec, threads);
  const int64_t grid = (int64_t)T * parts + ceil_div(rows, kZeroRows);
  if (k > 1 && (size_t)rows * vec * 16 >= kTokenMajorFrom && grid <= 0x7fffffff) {
    const int blocks = std::min(ceil_div(std::max(rows, T * k), 256), num_sms() * 4);
    const moe_status_t st = launch_k(positions_kernel, dim3(blocks), dim3(256), 0, s, ids, sid, T * k, E,
                                     rows, pos);
    if (st != MOE_OK) return st;
    return launch_k(permute_tokens_kernel, dim3((unsigned)grid), dim3(threads), 0, s, (const uint4*)x, sid,
                    (const int32_t*)pos, T, k, rows, vec, parts, (uint4*)xs);
  }
  const int blocks = std::min(ceil_div(rows, 8), num_sms() * 8);
  return launch_k(permute_kernel, dim3(blocks), dim3(256), 0, s, (const uint4*)x, ids, sid, T * k,
                  k, E, rows, vec, (uint4*)xs, pos);
}

moe_status_t launch_slot_sum(const void* ys, const int32_t* pos, const float* w, int T, int k,
                             int H, moe_dtype_t dt, int rows, void* out, cudaStream_t s) {
  const int vec = H * (int)dtype_size(dt) / 16;
  // rows shorter than a block's pieces get a smaller block
  const int threads = vec >= 256 ? 256 : std::max(32, ceil_div(vec, 32) * 32);
  const int parts = ceil_div(vec, threads);
  if ((int64_t)T * parts > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  auto go = [&](auto kern) {
    return launch_k(kern, dim3((unsigned)(T * parts)), dim3(threads), 0, s, (const uint4*)ys, pos,
                    w, k, rows, vec, parts, (uint4*)out);
  };
  if (dt == MOE_BF16)
    return w ? go(slot_sum_kernel<__nv_bfloat16, true>) : go(slot_sum_kernel<__nv_bfloat16, false>);
  return w ? go(slot_sum_kernel<float, true>) : go(slot_sum_kernel<float, false>);
}

moe_status_t launch_unpermute_backward(const void* dout, const void* ys, const int32_t* sid,
                                       const int32_t* pos, const float* w, int T, int k, int H,
                                       moe_dtype_t dt, int rows, void* dys, float* dw,
                                       cudaStream_t s) {
  const int vec = H * (int)dtype_size(dt) / 16;
  const dim3 grid((unsigned)(T + ceil_div(rows, kZeroRows)));
  const int threads = std::max(32, std::min(kUbThreads, ceil_div(vec, 32) * 32));
  if (dt == MOE_BF16)
    return launch_k(unpermute_backward_kernel<__nv_bfloat16>, grid, dim3(threads), 0, s,
                    (const uint4*)dout, (const uint4*)ys, sid, pos, w, T, k, rows, vec,
                    (uint4*)dys, dw);
  return launch_k(unpermute_backward_kernel<float>, grid, dim3(threads), 0, s,
                  (const uint4*)dout, (const uint4*)ys, sid, pos, w, T, k, rows, vec,
                  (uint4*)dys, dw);
}

}  // namespace moe
