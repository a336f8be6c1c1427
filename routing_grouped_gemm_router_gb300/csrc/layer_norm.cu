// layer_norm.cu — the layer norm, the residual join with dropout that takes the next layer norm in
// the same pass, and their gradients (moe_layer_norm, moe_dropout_join and their backward calls).
//
// With m = mean(x), r = (mean((x - m)^2) + eps)^-1/2, xn = (x - m) r, keep the mask over 1 - p:
//   norm   h = xn gamma + beta
//   join   out = x + scale keep y;  h = norm(out)
//   back   a = dh gamma:  d = dres + r (a - mean(a) - xn mean(a xn));  dx = d,  dy = scale keep d
//          dgamma = sum_t dh xn;  dbeta = sum_t dh
// Every row is read once and written once, so HBM bounds all of them, but where random numbers are drawn: the
// mask is computed from the element's number wherever it is needed, which takes a third of a join's
// instructions (116 of 336 for eight elements). The backward kernels' rows go through the rings and the column sums of row_ring.cuh.
// Measured, 8192 rows of bf16, us and TB/s: norm of 4096 channels 28.5 (4.7), of 7168 50 (4.7); its gradient with a
// residual 49 (5.5), 76.5 (6.1); join with the next norm 43.5 (6.2), 73 (6.5), with dropout 55 (4.9), 98 (4.8);
// its gradient with dropout 68 (4.9), 118.5 (5.0); dropout alone 27 (5.0), 46 (5.1). Of fp32, 4096 channels: 47 (5.7),
// 90 (5.9), 82 (6.5), 86 (6.2), 120.5 (5.6), 42 (6.4).
//
// The variance is summed about a mean that is already near the row's: a warp sums its own elements,
// then their squared distances from its own mean, and the warps' sums and distances are joined by
//   M2 = sum_w M2_w + n_w (m_w - m)^2.
// That takes two rounds of shuffles and one barrier a row, where a mean first and the squares after
// take two, and it loses nothing for rows whose mean is large against their spread, where a
// difference of squares would.
#include "row_ring.cuh"
#include "stack.cuh"

namespace moe {
namespace lnorm {

using namespace rows;

// ------------------------------------------------------------------- forward
// Keeps or drops eight elements and scales them: y * factor, or 0 whatever y is. ADDED: something is added to the
// result. The product then has to be rounded first, as dropout alone stores it, and the selection comes
// behind it: the compiler joins a packed product with a packed sum that follows it. (Behind the product it
// costs the join 54.4 -> 54.9 us at 8192 x 4096 in bf16; its gradient, which adds nothing, 118 -> 120 at x 7168.)
template <bool DROP, bool ADDED>
__device__ __forceinline__ void drop_scale(F2 (&y)[4], Philox* rng, const Drop& d, int64_t first) {
  if (DROP) {
    uint32_t w[8];
    rng->eight(first, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      split(ADDED ? y[i] * dup(d.factor) : y[i], lo, hi);
      y[i] = f2(w[2 * i] >= d.below ? lo : 0.f, w[2 * i + 1] >= d.below ? hi : 0.f);
      if (!ADDED) y[i] = y[i] * dup(d.factor);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = y[i] * dup(d.factor);
  }
}

// Rows of the forward kernel: `warps` warps a row, chunk c of the row held by thread c % (32 warps); several
// rows a CTA where one warp takes a row.
struct Rows {
  int T, H, chunks, warps;
  float eps, inv_h;
};

// JOIN: out = x + scale dropout(y), then (if gamma) its norm; otherwise the norm of x. A row's elements are all
// asked for at once and stay in registers, and a CTA is done after its row: with many small CTAs an SM has
// enough rows in flight to hide the chain of a row's reductions. (With persistent CTAs and the
// rings of the backward kernels three rows an SM were in flight, and 8192 rows of 4096 took 36 us.)
// THREADS, CTAS: of a CTA at most, and at least an SM where that is not 0. The join of bf16 rows in four chunks a
// thread is held to 72 registers: 8192 x 4096 55 us, with 92 as the compiler likes it 56.5.
template <typename T, int VPT, int THREADS, int CTAS, bool JOIN, bool DROP>
__global__ void __launch_bounds__(THREADS, CTAS)
    forward_kernel(const __grid_constant__ Rows R, const __grid_constant__ LayerArgs A) {
  __shared__ float near_mean[16], near_m2[16];
  const int group = R.warps * 32, local = threadIdx.x / group, g = threadIdx.x - local * group;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / group) + local;
  pdl_wait();
  pdl_trigger();
  if (t >= R.T) return;  // a warp with a row of its own
  const int64_t row = t * R.H;
  const uint8_t* from = (const uint8_t*)(JOIN ? A.y : A.x) + row * sizeof(T);
  const uint8_t* from_x = (const uint8_t*)A.x + row * sizeof(T);
  Chunk<T> q[VPT], xq[JOIN ? VPT : 1];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = g + v * group;
    if (c >= R.chunks) break;
    q[v].load(from + c * Chunk<T>::kBytes);
    if (JOIN) xq[v].load(from_x + c * Chunk<T>::kBytes);
  }
  Philox rng = DROP ? Philox(A.drop) : Philox();
  // The row stays as it is stored where that takes half the registers: more rows in flight for two more
  // conversions (norm of 8192 x 4096 32 -> 28.5 us, join without dropout 46 -> 43).
  constexpr bool PACKED = sizeof(T) == 2;
  F2 wide[PACKED ? 1 : VPT][4], s = dup(0.f);
  auto piece = [&](int v, F2 (&o)[4]) {
    if constexpr (PACKED) {
      q[v].get(o);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = wide[v][i];
    }
  };
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = g + v * group;
    if (c >= R.chunks) break;
    F2 o[4];
    q[v].get(o);
    if (JOIN) {
      F2 x[4];
      xq[v].get(x);
      if (DROP) drop_scale<DROP, true>(o, &rng, A.drop, row + c * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = DROP ? o[i] + x[i] : fma2(o[i], dup(A.drop.factor), x[i]);
      Chunk<T> out;
      out.set(o);
      out.store(A.out, row + c * 8);
      out.get(o);  // the norm reads what is stored
      if constexpr (PACKED) q[v] = out;
    }
    if constexpr (!PACKED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) wide[v][i] = o[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s = s + o[i];
  }
  if (JOIN && !A.gamma) return;
  // a warp's own mean, and the sum of squares about it
  const int full = R.chunks / group * 256, rest = R.chunks % group * 8;
  auto elements = [&](int w) { return (float)(full + min(max(rest - w * 256, 0), 256)); };
  float mean = warp_total(both(s)) / fmaxf(elements(g >> 5), 1.f);
  const F2 near = dup(-mean);
  s = dup(0.f);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if (g + v * group >= R.chunks) break;
    F2 o[4];
    piece(v, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 d = o[i] + near;
      s = fma2(d, d, s);
    }
  }
  float m2 = warp_total(both(s));
  if (R.warps > 1) {
    if ((threadIdx.x & 31) == 0) {
      near_mean[g >> 5] = mean;
      near_m2[g >> 5] = m2;
    }
    __syncthreads();
    mean = m2 = 0.f;
    for (int w = 0; w < R.warps; ++w) mean = fmaf(elements(w) * R.inv_h, near_mean[w], mean);
    for (int w = 0; w < R.warps; ++w) {
      const float off = near_mean[w] - mean;
      m2 += fmaf(elements(w) * off, off, near_m2[w]);
    }
  }
  const float r = rsqrtf(m2 * R.inv_h + R.eps);
  if (g == 0) {
    A.mean[t] = mean;
    A.rstd[t] = r;
  }
  const F2 rr = dup(r), mm = dup(-mean);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = g + v * group;
    if (c >= R.chunks) break;
    F2 ga[4], be[4], o[4];
    piece(v, o);
    load_w(A.gamma, c * 8, ga);
    if (A.beta) load_w(A.beta, c * 8, be);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 xn = (o[i] + mm) * rr;
      ga[i] = A.beta ? fma2(xn, ga[i], be[i]) : xn * ga[i];
    }
    Chunk<T> h;
    h.set(ga);
    h.store(A.h, row + c * 8);
  }
}

// ------------------------------------------------------------------- backward
// Sums of N values (2 or 4) over a row's group, in every thread of it, as group_sum: but a warp's lanes
// divide the values among them, so that 4 values take 6 rounds of shuffles and not 20, and as many again
// over the warps.
template <int N>
__device__ __forceinline__ void divided_sum(float (&v)[N], int group, Reducer& red, int& turn) {
  constexpr int LANES = 32 / N;  // that hold one value in the end
  const int lane = threadIdx.x & 31, which = lane / LANES;
#pragma unroll
  for (int off = 16, n = N / 2; n > 0; off >>= 1, n >>= 1) {
    const bool upper = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = upper ? v[i + n] : v[i], send = upper ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  float s = v[0];
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (group > 32) {
    const int warp = threadIdx.x >> 5, w = group >> 5, first = warp / w * w, j = lane % LANES;
    auto& buf = red.buf[turn];
    turn ^= 1;
    if (j == 0) buf[which][warp] = s;
    __syncthreads();
    s = j < w ? buf[which][first + j] : 0.f;
    if (LANES < 16 && j + LANES < w) s += buf[which][first + j + LANES];
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, s, i * LANES);
}

// JOIN: dy too. Row tensors: dh, x, (dres). A group takes ROWS rows at a time, whose sums meet at one barrier
// and whose weights are loaded once; dh and x stay in registers as they are stored, dres is read from
// the ring when the sums are there. FLAT (see Ring): no branch between a unit's rows and chunks, whose
// instructions then interleave.
template <typename T, int VPT, int THREADS, int ROWS, bool FLAT, bool JOIN, bool DROP>
__global__ void __launch_bounds__(THREADS, VPT <= 2 && THREADS <= 256 ? 2 : 1)
    backward_kernel(const __grid_constant__ Shape S, const __grid_constant__ LayerArgs A, int kinds,
                    const Outs outs) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Reducer red;
  const int local = threadIdx.x / S.group, g = threadIdx.x - local * S.group;
  Ring<T, VPT, 3, ROWS, FLAT> ring(S, smem, local, g);
  pdl_wait();
  pdl_trigger();
  ring.start();
  Philox rng = DROP ? Philox(A.drop) : Philox();
  int turn = 0;
  const bool res = A.dres;
  const F2 zero = dup(0.f);
  F2 sg[VPT][4], sb[VPT][4];
#pragma unroll
  for (int v = 0; v < VPT; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) sg[v][i] = sb[v][i] = zero;

  // a row's scalars are asked for one unit ahead: nothing else hides their way from L2. FLAT: 0 for rows behind
  // the last and threads that hold no chunk, whose xn has to be 0 and not (0 - mean) * rstd of some row.
  float m_next[ROWS], r_next[ROWS];
  auto scalars = [&](int64_t u) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      int64_t t = (u * S.per + local) * ROWS + r;
      const bool some = !FLAT || (t < S.T && (VPT > 1 || ring.has[0]));
      if (t >= S.T) t = 0;
      m_next[r] = some ? __ldg(A.mean_in + t) : 0.f;
      r_next[r] = some ? __ldg(A.rstd_in + t) : 0.f;
    }
  };
  scalars(blockIdx.x);
  F2 w[VPT][4];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[v][i] = zero;
    if (ring.has[v]) load_w(A.gamma, (g + v * S.group) * 8, w[v]);
  }
  for (int u = blockIdx.x; u < S.units; u += gridDim.x) {
    const int t0 = (u * S.per + local) * ROWS;
    F2 rr[ROWS], mm[ROWS];
    float rstd[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      rstd[r] = r_next[r];
      rr[r] = dup(rstd[r]);
      mm[r] = dup(-m_next[r]);
    }
    scalars((int64_t)u + gridDim.x);
    ring.wait();
    Chunk<T> xq[ROWS][VPT], dq[ROWS][VPT];
    F2 s1[ROWS], s2[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s1[r] = s2[r] = zero;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (!FLAT && !ring.has[v]) continue;
      const F2(&ga)[4] = w[v];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (!FLAT && t0 + r >= S.T) continue;
        ring.get(dq[r][v], 0, v, t0 + r, r);
        ring.template get<VPT == 1>(xq[r][v], 1, v, t0 + r, r);  // two chunks a thread: every one has its first
        F2 x[4], d[4];
        dq[r][v].get(d);
        xq[r][v].get(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 xn = (x[i] + mm[r]) * rr[r];
          sg[v][i] = fma2(d[i], xn, sg[v][i]);
          sb[v][i] = sb[v][i] + d[i];
          d[i] = d[i] * ga[i];
          s1[r] = fma2(d[i], xn, s1[r]);
          s2[r] = s2[r] + d[i];
        }
      }
    }
    float s[2 * ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      s[2 * r] = both(s1[r]);
      s[2 * r + 1] = both(s2[r]);
    }
    divided_sum<2 * ROWS>(s, S.group, red, turn);
    // dx = dres + r (a - mean(a) - mean(a xn) xn)
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = g + v * S.group;
      if (!FLAT && !ring.has[v]) continue;
      const F2(&ga)[4] = w[v];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (!FLAT && t0 + r >= S.T) continue;
        const F2 m1 = dup(-s[2 * r] * S.inv_h), m0 = dup(-s[2 * r + 1] * S.inv_h);
        const int64_t at = (int64_t)(t0 + r) * S.H + c * 8;
        F2 x[4], d[4];
        dq[r][v].get(d);
        xq[r][v].get(x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 xn = (x[i] + mm[r]) * rr[r];
          d[i] = fma2(xn, m1, fma2(d[i], ga[i], m0));
        }
        Chunk<T> o;
        if (res) {
          F2 f[4];
          ring.get(o, 2, v, t0 + r, r);
          o.get(f);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = fma2(d[i], rr[r], f[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = d[i] * rr[r];
        }
        const bool live = !FLAT || (t0 + r < S.T && ring.has[v]);
        o.set(d);
        if (live) o.store(A.dx, at);
        if (JOIN) {
          drop_scale<DROP, false>(d, &rng, A.drop, at);
          o.set(d);
          if (live) o.store(A.dy, at);
        }
      }
    }
    ring.refill(u);
  }
  leave_columns<VPT>(S, smem, local, g, sg, 0, kinds, 1.f, A.ws, outs);
  if (kinds > 1) leave_columns<VPT>(S, smem, local, g, sb, 1, kinds, 1.f, A.ws, outs);
}

// Chunks of 8 elements a thread holds. Backward, two: the sums over tokens take 16 registers a chunk. One for the
// norm alone where that was quicker; one and two, us in a graph (the join's gradient, longer in a thread,
// loses: 8192 x 4096 76 and 69):
//   rows                 200         400         800        1216        2432        4864   of channels
//   1000 bf16        6.3  5.9    7.7  6.7    7.5  8.3    7.7  8.0   11.1 11.4   14.9 15.9
//        fp32        6.4  6.2    8.0  7.2    8.9 10.0   10.6 10.9   14.4 14.7   20.9 19.6
//   2056 bf16        7.2  7.2    6.7  9.5    9.6 11.3   11.4 12.8   16.2 17.3   25.9 22.6
//        fp32        8.0  8.0    8.5 11.4   12.0 14.8   14.0 17.1   20.7 22.3   34.4 37.7
//   4096 bf16        7.7  9.0    9.5 10.3   13.5 13.7   15.4 15.7   21.6 20.7   33.7 32.5
//        fp32        9.5 11.2   12.9 13.4   17.7 17.9   21.7 19.8   34.5 32.3   58.8 56.9
// Two CTAs fit an SM. In two chunks a thread, rows of 129 to 288 chunks give them 3 to 6 warps each, in one 5 to
// 9. Shorter rows fill a CTA either way, several at once: one chunk a thread halves the rows of a CTA, which helps
// once every SM has some. Longer ones leave one CTA an SM: only while that one has few rows.
static bool one_chunk(const moe_layer_t& c) {
  const int chunks = c.H / 8, sms = num_sms();
  if (chunks <= 128) return c.T >= 8 * sms && c.T <= 16 * sms;
  if (chunks <= 288) return c.T <= 16 * sms;
  return chunks <= 512 && c.T > sms && c.T <= 3 * sms;
}
static int wide(const moe_layer_t& c, bool join) {
  const int chunks = c.H / 8;
  if (!join && one_chunk(c)) return 1;
  const int two = c.dtype == MOE_F32 ? 896 : 1024;
  return chunks <= 32 ? 1 : chunks <= two ? 2 : chunks <= 2048 ? 4 : 8;
}
// Forward, four, or eight for long rows, so that few warps share a row's reductions (8192 rows of bf16, four and
// eight, us: norm of 4096 28.5 and 29.5, of 7168 51.5 and 49.5; join 55 and 58, 126 and 97; join without dropout
// 43 and 46, 72 and 76, at every length). With few rows for an SM as few as give a row 512 threads at most:
// one row's latency counts.
static int narrow(const moe_layer_t& c, bool join, bool drop) {
  const int chunks = c.H / 8;
  if (c.T < 4 * num_sms()) return chunks <= 32 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8;
  const int four = c.dtype == MOE_F32 || (join && !drop) ? 2048 : 640;
  return chunks <= 32 ? 1 : chunks <= 64 ? 2 : chunks <= four ? 4 : 8;
}
static Shape shape_of(const moe_layer_t& c, int vec, int rows) {
  Shape s{};
  s.T = c.T;
  s.H = c.H;
  s.chunks = c.H / 8;
  s.group = ceil_div(ceil_div(s.chunks, vec), 32) * 32;
  s.rows = rows;
  s.per = std::min(ceil_div(c.T, rows), std::max(1, 256 / s.group));
  s.units = ceil_div(c.T, s.per * rows);
  s.scale = c.scale;
  s.eps = c.eps;
  s.inv_h = 1.0f / (float)c.H;
  return s;
}
// Rows that a group takes at a time in the backward kernels: two of bf16 for the norm alone, where that
// leaves every SM work; with the join's second gradient and its random numbers registers are better spent
// on one row without branches (8192 x 4096 69 and 75 us, 8192 x 7168 118 and 128; the norm alone of 7168
// 81 with one row and 77 with two).
static int rows_of(const moe_layer_t& c, bool join) {
  if (join || c.dtype != MOE_BF16 || c.H > 8192) return 1;
  return shape_of(c, wide(c, join), 2).units >= 2 * num_sms() ? 2 : 1;
}

using bf = __nv_bfloat16;

// Calls f with the instance of a dtype and a row length: element type, chunks and threads.
template <typename T_, int VPT, int THREADS>
struct Instance {
  using T = T_;
  static constexpr int vpt = VPT, threads = THREADS;
};
template <typename F>
static moe_status_t pick(const moe_layer_t& c, int v, int group, F f) {
  if (c.dtype == MOE_BF16) {
    if (v == 1) return group <= 256 ? f(Instance<bf, 1, 256>{}) : f(Instance<bf, 1, 512>{});
    if (v == 2)
      return group <= 256 ? f(Instance<bf, 2, 256>{}) : group <= 448 ? f(Instance<bf, 2, 448>{}) : f(Instance<bf, 2, 512>{});
    return v == 4 ? f(Instance<bf, 4, 512>{}) : f(Instance<bf, 8, 512>{});
  }
  if (v == 1) return group <= 256 ? f(Instance<float, 1, 256>{}) : f(Instance<float, 1, 512>{});
  if (v == 2) return group <= 256 ? f(Instance<float, 2, 256>{}) : f(Instance<float, 2, 448>{});
  return v == 4 ? f(Instance<float, 4, 512>{}) : f(Instance<float, 8, 512>{});
}

template <bool JOIN, bool DROP>
static moe_status_t forward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  const int v = narrow(c, JOIN, DROP);
  Rows R{c.T, c.H, c.H / 8, ceil_div(c.H / 8, 32 * v), c.eps, 1.0f / (float)c.H};
  const int per = R.warps == 1 ? 4 : 1;
  auto go = [&](auto kern) {
    return launch_k(kern, dim3(ceil_div(c.T, per)), dim3(R.warps * 32 * per), 0, s, (const Rows&)R, a);
  };
  auto with = [&](auto i) {
    using I = decltype(i);
    using T = typename I::T;
    if constexpr (JOIN && DROP && sizeof(T) == 2 && I::vpt == 4)
      if (R.warps * 32 * per <= 160) return go(forward_kernel<T, 4, 160, 5, JOIN, DROP>);
    return go(forward_kernel<T, I::vpt, 512, 0, JOIN, DROP>);
  };
  if (c.dtype == MOE_BF16)
    return v == 1   ? with(Instance<bf, 1, 512>{})
           : v == 2 ? with(Instance<bf, 2, 512>{})
           : v == 4 ? with(Instance<bf, 4, 512>{})
                    : with(Instance<bf, 8, 512>{});
  return v == 1   ? with(Instance<float, 1, 512>{})
         : v == 2 ? with(Instance<float, 2, 512>{})
         : v == 4 ? with(Instance<float, 4, 512>{})
                  : with(Instance<float, 8, 512>{});
}

// Bytes of rows in flight an SM in the backward kernels: with two rows a group, two stages of two CTAs.
constexpr size_t kBackBudget = 200 * 1024;

template <bool JOIN, bool DROP>
static moe_status_t backward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  Shape S = shape_of(c, wide(c, JOIN), rows_of(c, JOIN));
  S.in[S.n_in++] = a.dh;
  S.in[S.n_in++] = a.x;
  if (a.dres) S.in[S.n_in++] = a.dres;
  Outs outs{};
  int kinds = 0;
  outs.p[kinds++] = a.dgamma;
  if (a.dbeta) outs.p[kinds++] = a.dbeta;
  // the CTA's groups meet in shared memory at the end
  const size_t least = S.per > 1 ? (size_t)S.per * S.H * sizeof(float) : 0;
  int blocks = 0;
  const moe_status_t st = pick(c, wide(c, JOIN), S.group, [&](auto i) {
    using I = decltype(i);
    using T = typename I::T;
    auto go = [&](auto kern) {
      return run_within(kBackBudget, kern, S, sizeof(T), least, kRinged<T, I::vpt>, kMaxCtas, blocks, s, a, kinds,
                        outs);
    };
    if constexpr (I::vpt <= 2) {
      if constexpr (sizeof(T) == 2 && !JOIN)  // two rows of two chunks without branches: too many registers
        if (S.rows == 2) return go(backward_kernel<T, I::vpt, I::threads, 2, I::vpt == 1, JOIN, DROP>);
      return go(backward_kernel<T, I::vpt, I::threads, 1, true, JOIN, DROP>);
    } else {
      return go(backward_kernel<T, I::vpt, I::threads, 1, false, JOIN, DROP>);
    }
  });
  if (st != MOE_OK || blocks == 1) return st;
  return launch_column_sum(a.ws, blocks, kinds, c.H, outs, s);
}

}  // namespace lnorm

using namespace lnorm;

size_t layer_ws_bytes(const moe_layer_t& c) {
  // the same size for both kinds of call
  auto blocks_of = [&](bool join) { return rows::max_blocks(shape_of(c, wide(c, join), rows_of(c, join))); };
  const int blocks = std::max(blocks_of(false), blocks_of(true));
  return (size_t)blocks * 2 * c.H * sizeof(float);
}

moe_status_t launch_layer_norm(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  return forward<false, false>(c, a, s);
}
moe_status_t launch_layer_norm_backward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  return backward<false, false>(c, a, s);
}
moe_status_t launch_dropout_join(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  return a.drop.below ? forward<true, true>(c, a, s) : forward<true, false>(c, a, s);
}
moe_status_t launch_dropout_join_backward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s) {
  return a.drop.below ? backward<true, true>(c, a, s) : backward<true, false>(c, a, s);
}

// ------------------------------------------------------------------- dropout alone
namespace lnorm {

constexpr int kAhead = 4;  // pieces of 8 elements a thread has in flight

// Reads and writes each element once; the generator's multiplications keep the multiplier pipe 73 % busy.

template <typename T, bool DROP>
__global__ void __launch_bounds__(256) dropout_kernel(const uint8_t* x, void* out, int64_t pieces,
                                                      const __grid_constant__ Drop D) {
  pdl_wait();
  pdl_trigger();
  const int64_t first = (int64_t)blockIdx.x * (256 * kAhead) + threadIdx.x;
  Chunk<T> q[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (first + i * 256 < pieces) q[i].load(x + (first + i * 256) * Chunk<T>::kBytes);
  Philox rng = DROP ? Philox(D) : Philox();
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int64_t at = first + i * 256;
    if (at >= pieces) break;
    F2 v[4];
    q[i].get(v);
    drop_scale<DROP, false>(v, &rng, D, at * 8);
    q[i].set(v);
    q[i].store(out, at * 8);
  }
}

}  // namespace lnorm

moe_status_t launch_dropout(const moe_layer_t& c, const Drop& d, const void* x, void* out,
                            cudaStream_t s) {
  const int64_t pieces = (int64_t)c.T * (c.H / 8);
  const int64_t blocks = ceil_div64(pieces, 256 * kAhead);
  if (blocks > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  auto go = [&](auto kern) {
    return launch_k(kern, dim3((unsigned)blocks), dim3(256), 0, s, (const uint8_t*)x, out, pieces, d);
  };
  if (c.dtype == MOE_BF16) return d.below ? go(dropout_kernel<bf, true>) : go(dropout_kernel<bf, false>);
  return d.below ? go(dropout_kernel<float, true>) : go(dropout_kernel<float, false>);
}

}  // namespace moe
