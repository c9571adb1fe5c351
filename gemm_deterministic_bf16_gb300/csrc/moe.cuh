// moe.cuh -- the routing of one token, shared by the mixture-of-experts kernels.
#pragma once

#include "moe.h"

namespace detffn {

// Order of logits as unsigned keys: larger first, a NaN before all (it then
// shows in the weights), -0 equal to +0.  No key is 0 or the largest number.
__device__ __forceinline__ uint32_t moe_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return l != l ? 0xFFFFFFFEu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
// The logit of a key (a NaN for a NaN's).
__device__ __forceinline__ float moe_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// The keys of token q for moe_choose: lane l holds experts l, l + 32, ..., E <=
// 32 N (0: no such expert, or no such token).
template <int N>
__device__ __forceinline__ void moe_keys(const float* logits, int T, int E, int q, int lane, uint32_t (&key)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    key[i] = q < T && lane + 32 * i < E ? moe_key(__ldcg(logits + (long long)q * E + lane + 32 * i)) : 0u;
}

// The k experts of B tokens and their logits, by one warp; lane j ends with
// choice j of each.  A round takes the largest key, the lowest expert among
// equals: every lane keeps its own best, and the lane that held the winner
// finds its next.  The tokens' rounds run side by side, as each is a chain of
// exchanges that mostly waits.
struct MoeChoice {
  int expert;
  float logit;
};
template <int N, int B>
__device__ __forceinline__ void moe_choose(const uint32_t (&key)[B][N], int k, int lane, MoeChoice (&choice)[B]) {
  unsigned used[B];
  uint32_t best[B], mine[B];
  int at[B];
  auto next = [&](int b) {
    best[b] = 0;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (!(used[b] >> i & 1) && key[b][i] != 0 && key[b][i] >= best[b]) {
        best[b] = key[b][i];
        at[b] = i;
      }
  };
#pragma unroll
  for (int b = 0; b < B; ++b) {
    used[b] = mine[b] = 0;
    at[b] = 0;
    choice[b].expert = 0;
    next(b);
  }
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t high[B];
    int e[B];
#pragma unroll
    for (int b = 0; b < B; ++b) high[b] = __reduce_max_sync(0xffffffffu, best[b]);
#pragma unroll
    for (int b = 0; b < B; ++b)
      e[b] = (int)__reduce_min_sync(0xffffffffu, best[b] == high[b] ? (unsigned)(lane + 32 * at[b]) : 0x7FFFu);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (lane == (e[b] & 31)) {
        used[b] |= 1u << (e[b] >> 5);
        next(b);
      }
      if (lane == j) {
        mine[b] = high[b];
        choice[b].expert = e[b];
      }
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) choice[b].logit = moe_logit(mine[b]);
}

// Sum over all experts of exp(logit - top), by one warp.
__device__ __forceinline__ float moe_sum(const float* logits, int E, float top, int lane) {
  float s = 0.0f;
  for (int e = lane; e < E; e += 32) s += expf(__ldcg(logits + e) - top);
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// The weight of choice j of a token whose chosen logits are l[0 .. k - 1]
// (the first the largest): over the sum of the chosen where `all` is negative.
__device__ __forceinline__ float moe_weight(const float* l, int k, int j, float all) {
  const float top = l[0];
  float s = 0.0f;
  if (all < 0.0f) {
    for (int i = 0; i < k; ++i) s += expf(l[i] - top);
  } else {
    s = all;
  }
  return expf(l[j] - top) / s;
}

}  // namespace detffn
