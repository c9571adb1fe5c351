// k_moe.cu -- a mixture-of-experts layer for a few tokens: the router and the
// kernels that take any sizes.
//
//   l[t, e] = x[t, :] . Wr[e, :]                       (router logits, FP32)
//   the k largest of l[t, :] in descending order, the lowest index first among equals
//   w[t, j] = exp(l_j - max) / sum                     (the sum over the k chosen, or over all E)
//   h = SiLU(x Wg[e]^T) * (x Wu[e]^T),  y = h Wd[e]^T  (the expert, FP32 sums, h rounded once)
//   out[t, :] = sum over j = 0 .. k-1 of w[t, j] y[t, j, :]
//
// Every sum runs in an order that the sizes H and I alone fix, so a token's
// result does not depend on the other tokens of the call.
#include "elt.cuh"
#include "moe.h"

namespace detffn {
namespace {

// Sum over k of a[k] b[k], by one warp: lane l takes k = l, l + 32, ...
template <int DT>
__device__ __forceinline__ float warp_dot(const typename Io<DT>::E* a, const typename Io<DT>::E* b, long long K,
                                          int lane) {
  float s = 0.0f;
  for (long long k = lane; k < K; k += 32) s = fmaf(Io<DT>::ld(a + k), Io<DT>::ld(b + k), s);
  return warp_sum(s);
}

// Logits of expert blockIdx.x: one warp per token.
template <int DT>
__global__ void __launch_bounds__(256) k_logits(const __grid_constant__ MoeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x;
  for (int t = warp; t < a.T; t += 8) {
    const float l = warp_dot<DT>(static_cast<const E*>(a.x) + t * a.H, static_cast<const E*>(a.Wr) + e * a.H, a.H, lane);
    if (lane == 0) a.logits[t * a.E + e] = l;
  }
}

// Order of logits: larger first, a NaN before all (it then shows in the
// weights), the lower index first among equals.
__device__ __forceinline__ unsigned long long rank_key(float l, int e) {
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 becomes +0
  const uint32_t k = l != l ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return ((unsigned long long)k << 32) | (uint32_t)~e;
}

// The choice of one token by one warp; E <= 512 logits, 16 a lane.
__device__ void choose(const float* logits, int E, int k, bool normalize, int lane, int* experts, float* weights) {
  constexpr int N = kMoeMaxExperts / 32;
  float l[N];
  unsigned used = 0;
  float top = -INFINITY, all = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? logits[e] : -INFINITY;
  }
  float w = 0.0f, sum = 0.0f;
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    unsigned long long best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !(used >> i & 1)) {
        const unsigned long long q = rank_key(l[i], e);
        best = q > best ? q : best;
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, d);
      best = o > best ? o : best;
    }
    const int e = (int)~(uint32_t)best;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e == lane + 32 * i) {
        used |= 1u << i;
        v = l[i];
      }
    v = __shfl_sync(0xffffffffu, v, e & 31);
    if (j == 0) top = v;
    const float x = expf(v - top);
    sum += x;
    if (lane == j) {
      w = x;
      mine = e;
    }
  }
  if (!normalize) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 32 * i < E) all += expf(l[i] - top);
    sum = warp_sum(all);
  }
  if (lane < k) {
    experts[lane] = mine;
    weights[lane] = w / sum;
  }
}

// The choices of all tokens and the pairs ordered by expert, by one block.
__global__ void __launch_bounds__(1024) k_select(const __grid_constant__ MoeArgs a) {
  __shared__ int ids[kMoeMaxTokens * kMoeMaxTopK], count[kMoeMaxExperts + 1];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, P = a.T * a.k;
  for (int t = warp; t < a.T; t += blockDim.x / 32)
    choose(a.logits + (long long)t * a.E, a.E, a.k, a.normalize, lane, a.experts + t * a.k, a.weights + t * a.k);
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += blockDim.x) ids[p] = a.experts[p];
  __syncthreads();
  const int e = threadIdx.x;
  if (e < a.E) {
    int c = 0;
    for (int p = 0; p < P; ++p) c += ids[p] == e;
    count[e] = c;
  }
  __syncthreads();
  if (e < a.E) {
    int at = 0;
    for (int q = 0; q < e; ++q) at += count[q];
    a.first[e] = at;
    if (e == a.E - 1) a.first[a.E] = P;
    for (int p = 0; p < P; ++p)
      if (ids[p] == e) {
        a.pair[at] = p;
        a.pos[p] = at++;
      }
  }
}

// h of expert blockIdx.y: one warp per feature i of I.
template <int DT>
__global__ void __launch_bounds__(256) k_gateup(const __grid_constant__ MoeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  const long long i = blockIdx.x * 8ll + warp;
  if (i >= a.I) return;
  const int p0 = a.first[e], p1 = a.first[e + 1];
  const E* wg = static_cast<const E*>(a.Wg) + (e * a.I + i) * a.H;
  const E* wu = static_cast<const E*>(a.Wu) + (e * a.I + i) * a.H;
  for (int p = p0; p < p1; ++p) {
    const E* x = static_cast<const E*>(a.x) + (a.pair[p] / a.k) * a.H;
    const float g = warp_dot<DT>(x, wg, a.H, lane), u = warp_dot<DT>(x, wu, a.H, lane);
    if (lane == 0) Io<DT>::st(static_cast<E*>(a.h) + p * a.I + i, g / (1.0f + expf(-g)) * u);
  }
}

// out of token blockIdx.y: one warp per feature r of H.
template <int DT>
__global__ void __launch_bounds__(256) k_down(const __grid_constant__ MoeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.y;
  const long long r = blockIdx.x * 8ll + warp;
  if (r >= a.H) return;
  float s = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int q = t * a.k + j;
    const E* w = static_cast<const E*>(a.Wd) + (a.experts[q] * a.H + r) * a.I;
    s = fmaf(a.weights[q], warp_dot<DT>(static_cast<const E*>(a.h) + a.pos[q] * a.I, w, a.I, lane), s);
  }
  if (lane == 0) Io<DT>::st(static_cast<E*>(a.out) + t * a.H + r, s);
}

template <int DT>
cudaError_t general(const MoeArgs& a, cudaStream_t st) {
  cudaError_t e = launch_dependent(k_logits<DT>, dim3(a.E), 256, 0, st, a);
  if (e == cudaSuccess) e = launch_dependent(k_select, dim3(1), 1024, 0, st, a);
  if (e == cudaSuccess) e = launch_dependent(k_gateup<DT>, dim3((unsigned)((a.I + 7) / 8), a.E), 256, 0, st, a);
  if (e == cudaSuccess) e = launch_dependent(k_down<DT>, dim3((unsigned)((a.H + 7) / 8), a.T), 256, 0, st, a);
  return e;
}

}  // namespace

cudaError_t launch_moe_general(const MoeArgs& a, cudaStream_t st) {
  return a.dtype == DETFFN_F32 ? general<DETFFN_F32>(a, st)
         : a.dtype == DETFFN_F16 ? general<DETFFN_F16>(a, st) : general<DETFFN_BF16>(a, st);
}

}  // namespace detffn
