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

// Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, 2011): four random numbers of a block's
// counter and the key. Two multiplications of 32 by 32 bits a round, four instructions after
// fusion of the exclusive-ors, so a number costs about as much as the arithmetic of a norm's element.
struct Philox {
  uint32_t k0, k1, s0, s1;
  __device__ __forceinline__ Philox() {}
  __device__ __forceinline__ explicit Philox(const Drop& d) {
    const uint64_t seed = (uint64_t)__ldg((const long long*)d.rng);
    const uint64_t stream = (uint64_t)__ldg((const long long*)d.rng + 1);
    k0 = (uint32_t)seed;
    k1 = (uint32_t)(seed >> 32);
    s0 = (uint32_t)stream;
    s1 = (uint32_t)(stream >> 32) + d.site;
  }
  __device__ __forceinline__ void block(uint64_t b, uint32_t (&r)[4]) const {
    uint32_t c0 = (uint32_t)b, c1 = (uint32_t)(b >> 32), c2 = s0, c3 = s1, a = k0, e = k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
      c0 = (uint32_t)(q >> 32) ^ c1 ^ a;
      c1 = (uint32_t)q;
      c2 = (uint32_t)(p >> 32) ^ c3 ^ e;
      c3 = (uint32_t)p;
      a += 0x9E3779B9u;
      e += 0xBB67AE85u;
    }
    r[0] = c0;
    r[1] = c1;
    r[2] = c2;
    r[3] = c3;
  }
  // of the eight elements from `first` on, a multiple of 8
  __device__ __forceinline__ void eight(int64_t first, uint32_t (&r)[8]) const {
    uint32_t a[4], b[4];
    block((uint64_t)first >> 2, a);
    block(((uint64_t)first >> 2) + 1, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = a[i];
      r[4 + i] = b[i];
    }
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
