// stack.cuh — internals of the operators around a stack's blocks (internal header): the random
// numbers of dropout, launch declarations.
#pragma once

#include "common.cuh"
#include "moe_stack.h"

namespace moe {

enum : int { kStatusBadOffsets = 5 };  // sequence offsets that decrease or leave [0, T]

// ------------------------------------------------------------------- random numbers
// Dropout as the kernels take it: elements whose number is below `below` are dropped, the others
// multiplied by `factor` (scale / (1 - p)).
struct Drop {
  const int64_t* rng;
  uint32_t below, site;
  float factor;
};

// Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, 2011): a round takes the counter c to
//   (hi(M1 c2) ^ c1 ^ k0, lo(M1 c2), hi(M0 c0) ^ c3 ^ k1, lo(M0 c0)),  the keys k a constant further.
// Here c = (b, b >> 32, stream, stream >> 32): all that does not depend on the low word of b is computed
// once (one product of the first round, one of the second), the round keys are kept in registers.
// A round is then two products and two exclusive-ors of three; with the keys' sums and all products in
// every round a join issued 34 instructions more for eight elements (336 now). A product keeps the
// multiplier pipe four cycles: 36 for eight elements are 144 of the 350 cycles that HBM leaves for a
// warp's eight elements a lane in a join of bf16 rows.
struct Philox {
  static constexpr uint32_t M0 = 0xD2511F53u, M1 = 0xCD9E8D57u;
  uint32_t key[8][2];  // of rounds 3 to 10
  uint32_t c0_1, c1k_2, k1s_1, k1_2;  // c0 after round 1 with a zero high word; what rounds 1 and 2 add
  uint32_t high, c2_2, c3_2;          // of the high word in `high`
  __device__ __forceinline__ Philox() {}
  __device__ __forceinline__ explicit Philox(const Drop& d) {
    const uint64_t seed = (uint64_t)__ldg((const long long*)d.rng);
    const uint64_t stream = (uint64_t)__ldg((const long long*)d.rng + 1);
    const uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    constexpr uint32_t W0 = 0x9E3779B9u, W1 = 0xBB67AE85u;
    const uint64_t q = (uint64_t)M1 * (uint32_t)stream;
    c0_1 = (uint32_t)(q >> 32) ^ k0;
    c1k_2 = (uint32_t)q ^ (k0 + W0);
    k1s_1 = ((uint32_t)(stream >> 32) + d.site) ^ k1;
    k1_2 = k1 + W1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      key[i][0] = k0 + (i + 2) * W0;
      key[i][1] = k1 + (i + 2) * W1;
      // opaque: kept, not added up again wherever it is used
      asm("" : "+r"(key[i][0]), "+r"(key[i][1]));
    }
    set_high(0);
  }
  __device__ __forceinline__ void set_high(uint32_t h) {
    high = h;
    const uint64_t p = (uint64_t)M0 * (c0_1 ^ h);
    c2_2 = (uint32_t)(p >> 32) ^ k1_2;
    c3_2 = (uint32_t)p;
  }
  __device__ __forceinline__ void block(uint32_t low, uint32_t* r) const {
    const uint64_t p = (uint64_t)M0 * low;                                   // round 1
    const uint64_t q = (uint64_t)M1 * ((uint32_t)(p >> 32) ^ k1s_1);         // round 2
    uint32_t c0 = (uint32_t)(q >> 32) ^ c1k_2, c1 = (uint32_t)q, c2 = c2_2 ^ (uint32_t)p, c3 = c3_2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t a = (uint64_t)M0 * c0, b = (uint64_t)M1 * c2;
      c0 = (uint32_t)(b >> 32) ^ c1 ^ key[i][0];
      c1 = (uint32_t)b;
      c2 = (uint32_t)(a >> 32) ^ c3 ^ key[i][1];
      c3 = (uint32_t)a;
    }
    r[0] = c0;
    r[1] = c1;
    r[2] = c2;
    r[3] = c3;
  }
  // of the eight elements from `first` on, a multiple of 8
  __device__ __forceinline__ void eight(int64_t first, uint32_t (&r)[8]) {
    const uint32_t h = (uint32_t)((uint64_t)first >> 34), low = (uint32_t)((uint64_t)first >> 2);
    if (h != high) set_high(h);
    block(low, r);
    block(low + 1, r + 4);  // low is even
  }
};

// ------------------------------------------------------------------- launches
struct LayerArgs {  // pointers of the layer norm's and the join's kernels
  const void *x, *y, *dh, *dres;
  const float *gamma, *beta, *mean_in, *rstd_in;
  void *out, *h, *dx, *dy;
  float *mean, *rstd, *dgamma, *dbeta;
  float* ws;
  Drop drop;
};
size_t layer_ws_bytes(const moe_layer_t& c);
moe_status_t launch_layer_norm(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s);
moe_status_t launch_layer_norm_backward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s);
moe_status_t launch_dropout_join(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s);
moe_status_t launch_dropout_join_backward(const moe_layer_t& c, const LayerArgs& a, cudaStream_t s);
moe_status_t launch_dropout(const moe_layer_t& c, const Drop& d, const void* x, void* out,
                            cudaStream_t s);

moe_status_t launch_embed(const void* tokens, bool wide, int T, const void* table, int V, int H,
                          moe_dtype_t dt, float scale, void* out, cudaStream_t s);
size_t embed_ws_bytes(int T, int V, int H);
moe_status_t launch_embed_backward(const void* dx, const void* tokens, bool wide, int T, int V, int H,
                                   moe_dtype_t dt, moe_dtype_t out_dt, float scale, int accumulate,
                                   void* dtable, void* ws, cudaStream_t s);

size_t balance_ws_bytes(const moe_balance_t& c);
moe_status_t launch_balance(const moe_balance_t& c, const float* logits, const int32_t* ids,
                            float* losses, int32_t* counts, int32_t* tokens, float* prob,
                            int32_t* totals, void* ws, cudaStream_t s);
moe_status_t launch_balance_backward(const moe_balance_t& c, const float* dlosses,
                                     const float* logits, const int32_t* counts,
                                     const int32_t* tokens, const int32_t* totals, int accumulate,
                                     float* dlogits, cudaStream_t s);
int balance_status_read(int reset);

}  // namespace moe
