// moe.cuh -- the routing of one token, shared by the mixture-of-experts kernels.
#pragma once

#include "moe.h"

namespace detffn {

// Order of logits as unsigned keys: larger first, a NaN before all (it then
// shows in the weights), -0 equal to +0.
__device__ __forceinline__ uint32_t moe_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return l != l ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
// The logit of a key (a NaN for a NaN's).
__device__ __forceinline__ float moe_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// The k experts of one token and their weights, by one warp; lane l holds the
// logits of experts l, l + 32, ..., E <= 32 N.  Each round takes the largest
// key, the lowest expert among equals: every lane keeps its own best, and the
// lane that held the winner finds its next.  Lane j ends with choice j.
struct MoeChoice {
  int expert;
  float weight;
};
template <int N>
__device__ __forceinline__ MoeChoice moe_choose(const float* logits, int E, int k, bool normalize, int lane) {
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = lane + 32 * i < E ? moe_key(__ldcg(logits + lane + 32 * i)) : 0u;
  unsigned used = 0;
  uint32_t best = 0, mine = 0;
  int at = 0, choice = 0;
  auto next = [&] {
    best = 0;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)   // (a valid key is never 0)
      if (!(used >> i & 1) && key[i] != 0 && key[i] >= best) {
        best = key[i];
        at = i;
      }
  };
  next();
  for (int j = 0; j < k; ++j) {
    const uint32_t high = __reduce_max_sync(0xffffffffu, best);
    const unsigned who = __ballot_sync(0xffffffffu, best == high);
    int e;
    if (__popc(who) == 1) {
      const int src = __ffs(who) - 1;
      e = src + 32 * __shfl_sync(0xffffffffu, at, src);
    } else {
      e = (int)__reduce_min_sync(0xffffffffu, best == high ? (unsigned)(lane + 32 * at) : 0x7FFFu);
    }
    if (lane == (e & 31)) {
      used |= 1u << (e >> 5);
      next();
    }
    if (lane == j) {
      mine = high;
      choice = e;
    }
  }
  const float l = moe_logit(mine), top = __shfl_sync(0xffffffffu, l, 0);
  const float x = lane < k ? expf(l - top) : 0.0f;
  float sum = x;
  if (!normalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] != 0) sum += expf(moe_logit(key[i]) - top);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return {choice, x / sum};
}

}  // namespace detffn
