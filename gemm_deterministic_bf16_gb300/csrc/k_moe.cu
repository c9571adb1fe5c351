// k_moe.cu -- a mixture-of-experts layer for a few tokens: the router and the
// kernels that take any sizes.
//
//   l[t, e] = x[t, :] . Wr[e, :]                       (router logits, FP32)
//   the k largest of l[t, :] in descending order, the lowest index first among equals
//   w[t, j] = exp(l_j - max) / sum                     (the sum over the k chosen, or over all E)
//   h = SiLU(x Wg[e]^T) * (x Wu[e]^T),  y = h Wd[e]^T  (the expert; FP32 sums, h in FP32 here)
//   out[t, :] = sum over j = 0 .. k-1 of w[t, j] y[t, j, :]
//
// Every sum runs in an order that the sizes H and I alone fix, so a token's
// result does not depend on the other tokens of the call.
#include "elt.cuh"
#include "moe.cuh"

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

// Router logits of four tokens and four experts by one block: each of eight
// warps takes an eighth of H (in 16-byte vectors; a token's sum is split by H
// alone), the sixteen sums of a warp meet in sixteen exchanges instead of
// eighty, and sixteen threads add the warps' parts in order.  What bounds it
// is the latency of its loads, so all of a warp's are independent.
// Block 0 also clears the counters of the kernel that follows.
template <int DT>
__global__ void __launch_bounds__(256) k_logits_tile(const __grid_constant__ MoeArgs a, int* counters, int n) {
  __shared__ float part[8][16];
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = blockIdx.x * 4, t0 = blockIdx.y * 4;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < n; i += blockDim.x) counters[i] = 0;
  const int vecs = (int)(a.H / 8), per = (vecs + 7) / 8, lo = warp * per, hi = min(vecs, lo + per);
  const E* x = static_cast<const E*>(a.x) + t0 * a.H;
  const E* w = static_cast<const E*>(a.Wr) + e0 * a.H;
  const int nt = min(4, a.T - t0), ne = min(4, a.E - e0);
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
#pragma unroll 2
  for (int c = lo + lane; c < hi; c += 32) {
    float p[4][8], q[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (past the last token or expert: the last one's, and its sum is not stored)
      Io<DT>::ld8(x + min(i, nt - 1) * a.H + 8 * c, p[i]);
      Io<DT>::ld8(w + min(i, ne - 1) * a.H + 8 * c, q[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i] = fmaf(p[i >> 2][j], q[i & 3][j], v[i]);
  }
  // Lane l keeps the half of the values that bit 0, 1, 2, 3 of l names in turn:
  // it ends with value l & 15 (bits reversed), then both halves of the warp add.
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int half = 8 >> b;
    const bool up = lane >> b & 1;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half];
      v[i] = (up ? v[i + half] : v[i]) + __shfl_xor_sync(0xffffffffu, send, 1 << b);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
  if (lane < 16) part[warp][((lane & 1) << 3) | ((lane & 2) << 1) | ((lane & 4) >> 1) | ((lane & 8) >> 3)] = v[0];
  __syncthreads();
  if (threadIdx.x < 16) {
    const int t = threadIdx.x >> 2, e = threadIdx.x & 3;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
    if (t < nt && e < ne) a.logits[(long long)(t0 + t) * a.E + e0 + e] = s;
  }
}

// The same for any H and alignment: expert blockIdx.x, one warp per token.
template <int DT>
__global__ void __launch_bounds__(256) k_logits(const __grid_constant__ MoeArgs a, int* counters, int n) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x;
  if (e == 0)
    for (int i = threadIdx.x; i < n; i += blockDim.x) counters[i] = 0;
  for (int t = warp; t < a.T; t += 8) {
    const float s = warp_dot<DT>(static_cast<const E*>(a.x) + t * a.H, static_cast<const E*>(a.Wr) + e * a.H, a.H, lane);
    if (lane == 0) a.logits[t * a.E + e] = s;
  }
}

// The choices of all tokens and the pairs ordered by expert, by one block.
__global__ void __launch_bounds__(1024) k_select(const __grid_constant__ MoeArgs a) {
  __shared__ int ids[kMoeMaxTokens * kMoeMaxTopK], count[kMoeMaxExperts + 1];
  __shared__ float chosen[kMoeMaxTokens * kMoeMaxTopK];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, P = a.T * a.k;
  for (int t = warp; t < a.T; t += blockDim.x / 32) {
    const float* l = a.logits + (long long)t * a.E;
    uint32_t key[1][kMoeMaxExperts / 32];
    MoeChoice chose[1];
    moe_keys<kMoeMaxExperts / 32>(a.logits, a.T, a.E, t, lane, key[0]);
    moe_choose<kMoeMaxExperts / 32, 1>(key, a.k, lane, chose);
    const MoeChoice c = chose[0];
    if (lane < a.k) {
      a.experts[t * a.k + lane] = c.expert;
      chosen[t * a.k + lane] = c.logit;
    }
    __syncwarp();
    const float all = a.normalize ? -1.0f : moe_sum(l, a.E, chosen[t * a.k], lane);
    if (lane < a.k) a.weights[t * a.k + lane] = moe_weight(chosen + t * a.k, a.k, lane, all);
  }
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
    if (lane == 0) static_cast<float*>(a.h)[p * a.I + i] = g / (1.0f + expf(-g)) * u;
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
    const float* hp = static_cast<const float*>(a.h) + a.pos[q] * a.I;
    float y = 0.0f;
    for (long long i = lane; i < a.I; i += 32) y = fmaf(Io<DT>::ld(w + i), hp[i], y);
    s = fmaf(a.weights[q], warp_sum(y), s);
  }
  if (lane == 0) Io<DT>::st(static_cast<E*>(a.out) + t * a.H + r, s);
}

template <int DT>
cudaError_t logits(const MoeArgs& a, int* counters, int n, cudaStream_t st) {
  const bool vec = a.H % 8 == 0 && (((uintptr_t)a.x | (uintptr_t)a.Wr) & 15u) == 0;
  if (vec) return launch_dependent(k_logits_tile<DT>, dim3((a.E + 3) / 4, (a.T + 3) / 4), 256, 0, st, a, counters, n);
  return launch_dependent(k_logits<DT>, dim3(a.E), 256, 0, st, a, counters, n);
}

template <int DT>
cudaError_t general(const MoeArgs& a, cudaStream_t st) {
  cudaError_t e = launch_moe_logits(a, nullptr, 0, st);
  if (e == cudaSuccess) e = launch_dependent(k_select, dim3(1), 1024, 0, st, a);
  if (e == cudaSuccess) e = launch_dependent(k_gateup<DT>, dim3((unsigned)((a.I + 7) / 8), a.E), 256, 0, st, a);
  if (e == cudaSuccess) e = launch_dependent(k_down<DT>, dim3((unsigned)((a.H + 7) / 8), a.T), 256, 0, st, a);
  return e;
}

}  // namespace

cudaError_t launch_moe_logits(const MoeArgs& a, int* counters, int n, cudaStream_t st) {
  return a.dtype == DETFFN_F32 ? logits<DETFFN_F32>(a, counters, n, st)
         : a.dtype == DETFFN_F16 ? logits<DETFFN_F16>(a, counters, n, st) : logits<DETFFN_BF16>(a, counters, n, st);
}

cudaError_t launch_moe_general(const MoeArgs& a, cudaStream_t st) {
  return a.dtype == DETFFN_F32 ? general<DETFFN_F32>(a, st)
         : a.dtype == DETFFN_F16 ? general<DETFFN_F16>(a, st) : general<DETFFN_BF16>(a, st);
}

}  // namespace detffn
