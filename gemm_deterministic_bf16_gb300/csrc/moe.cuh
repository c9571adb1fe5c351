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

// The k experts of one token and their logits, by one warp; lane l holds the
// keys of experts l, l + 32, ..., E <= 32 N (0: no such expert).  Each round takes the largest
// key, the lowest expert among equals: every lane keeps its own best, and the
// lane that held the winner finds its next.  Lane j ends with choice j.
struct MoeChoice {
  int expert;
  float logit;
};
template <int N>
__device__ __forceinline__ void moe_keys(const float* logits, int T, int E, int q, int lane, uint32_t (&key)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    key[i] = q < T && lane + 32 * i < E ? moe_key(__ldcg(logits + (long long)q * E + lane + 32 * i)) : 0u;
}
template <int N>
__device__ __forceinline__ MoeChoice moe_choose(const uint32_t (&key)[N], int k, int lane) {
  unsigned used = 0;
  uint32_t best = 0, mine = 0;
  int at = 0, choice = 0;
  auto next = [&] {
    best = 0;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (!(used >> i & 1) && key[i] != 0 && key[i] >= best) {
        best = key[i];
        at = i;
      }
  };
  next();
  for (int j = 0; j < k; ++j) {
    const uint32_t high = __reduce_max_sync(0xffffffffu, best);
    const int e = (int)__reduce_min_sync(0xffffffffu, best == high ? (unsigned)(lane + 32 * at) : 0x7FFFu);
    if (lane == (e & 31)) {
      used |= 1u << (e >> 5);
      next();
    }
    if (lane == j) {
      mine = high;
      choice = e;
    }
  }
  return {choice, moe_logit(mine)};
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
