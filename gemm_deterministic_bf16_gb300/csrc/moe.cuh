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
// lane that held the winner finds its next.
template <int N, class Id>
__device__ void moe_choose(const float* logits, int E, int k, bool normalize, int lane, Id* experts, float* weights) {
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = lane + 32 * i < E ? moe_key(logits[lane + 32 * i]) : 0u;
  unsigned used = 0;
  uint32_t best = 0;
  int at = 0x7FFF;
  auto mine = [&] {
    best = 0;
    at = 0x7FFF;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (lane + 32 * i < E && !(used >> i & 1) && key[i] >= best) {
        best = key[i];
        at = lane + 32 * i;
      }
  };
  mine();
  float top = 0.0f, w = 0.0f, sum = 0.0f;
  int choice = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t high = __reduce_max_sync(0xffffffffu, best);
    const int e = (int)__reduce_min_sync(0xffffffffu, best == high ? (unsigned)at : 0x7FFFu);
    if (e == at) {
      used |= 1u << (e >> 5);
      mine();
    }
    const float l = moe_logit(high);
    if (j == 0) top = l;
    const float x = expf(l - top);
    sum += x;
    if (lane == j) {
      w = x;
      choice = e;
    }
  }
  if (!normalize) {
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 32 * i < E) all += expf(moe_logit(key[i]) - top);
#pragma unroll
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    sum = all;
  }
  if (lane < k) {
    experts[lane] = (Id)choice;
    weights[lane] = w / sum;
  }
}

}  // namespace detffn
