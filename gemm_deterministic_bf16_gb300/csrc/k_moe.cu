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

// Sums over a warp of sixteen values of every lane, in sixteen exchanges instead
// of eighty: lane l keeps the half of the values that bit 0, 1, 2, 3 of l names
// in turn and ends with value sum16_of(l), then both halves of the warp add.
__device__ __forceinline__ int sum16_of(int lane) {
  return ((lane & 1) << 3) | ((lane & 2) << 1) | ((lane & 4) >> 1) | ((lane & 8) >> 3);
}
__device__ __forceinline__ float sum16(float (&v)[16], int lane) {
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
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// Router logits of four tokens and four experts by one block: each of eight
// warps takes an eighth of H (in 16-byte vectors; a token's sum is split by H
// alone), the sixteen sums of a warp meet in sixteen exchanges instead of
// eighty, and sixteen threads add the warps' parts in order.  What bounds it
// is the latency of its loads, so all of a warp's are independent (64 tokens of
// 64 experts, H = 4096: 54 us with a warp to a logit and its loads in turn; one
// token of 128, H = 2048: the next kernel, under way, waits 1.5 us for it).
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
  const float mine = sum16(v, lane);
  if (lane < 16) part[warp][sum16_of(lane)] = mine;
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

// N consecutive elements: one, four of FP32 or eight.
template <int DT, int N>
__device__ __forceinline__ void load_n(const typename Io<DT>::E* p, float (&f)[N]) {
  if constexpr (N == 8) {
    Io<DT>::ld8(p, f);
  } else if constexpr (N == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
  } else {
    f[0] = Io<DT>::ld(p);
  }
}

// Products of four rows of x (of type XT) with four rows of weights over K, by
// one warp: value 4 i + j is x_i . w_j.  VEC: 16-byte vectors of weights.
template <int DT, int XT, bool VEC>
__device__ __forceinline__ void tile16(const typename Io<XT>::E* const (&x)[4], const typename Io<DT>::E* const (&w)[4],
                                       long long K, int lane, float (&v)[16]) {
  constexpr int N = !VEC ? 1 : DT == DETFFN_F32 ? 4 : 8;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
#pragma unroll 2
  for (long long k = (long long)lane * N; k < K; k += 32 * N) {
    float a[4][N], b[4][N];
#pragma unroll
    for (int i = 0; i < 4; ++i) load_n<DT, N>(w[i] + k, b[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_n<XT, N>(x[i] + k, a[i]);
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) v[i] = fmaf(a[i >> 2][j], b[i & 3][j], v[i]);
  }
}

// What bounds the two kernels below is HBM for a few pairs of an expert and the
// L2 beyond: an expert's weights are read once for every four of its pairs.  A
// warp takes two features of gate and of up, or four of the output, so that
// what it loads of x serves sixteen sums (FP32, 64 tokens, 6 of 64 experts,
// H = 4096, I = 1536: 1538 us, and 7319 with one sum to a warp; 7 tokens, 2 of
// 16, I = 1416: 130 and 312, the weights alone take 101).

// h of expert blockIdx.y: features 2 i and 2 i + 1 by one warp.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) k_gateup(const __grid_constant__ MoeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  const long long i0 = 2 * (blockIdx.x * 8ll + warp), i1 = min(i0 + 1, a.I - 1);
  if (i0 >= a.I) return;
  const int p0 = a.first[e], p1 = a.first[e + 1];
  const E *wg = static_cast<const E*>(a.Wg) + e * a.I * a.H, *wu = static_cast<const E*>(a.Wu) + e * a.I * a.H;
  const E* const w[4] = {wg + i0 * a.H, wu + i0 * a.H, wg + i1 * a.H, wu + i1 * a.H};
  for (int p = p0; p < p1; p += 4) {
    const E* x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)   // (past the last pair: the last again)
      x[i] = static_cast<const E*>(a.x) + (a.pair[min(p + i, p1 - 1)] / a.k) * a.H;
    float v[16];
    tile16<DT, DT, VEC>(x, w, a.H, lane, v);
    // Lanes l and l + 8 hold gate and up of one feature and pair.
    const float g = sum16(v, lane), u = __shfl_xor_sync(0xffffffffu, g, 8);
    const int of = sum16_of(lane), q = p + (of >> 2), f = of >> 1 & 1;
    if (lane < 8 && q < p1 && i0 + f < a.I) static_cast<float*>(a.h)[q * a.I + i0 + f] = g * sigma<false>(g).s * u;
  }
}

// y of the pairs of expert blockIdx.y: features 4 r .. 4 r + 3 by one warp.
template <int DT, bool VEC>
__global__ void __launch_bounds__(256) k_down(const __grid_constant__ MoeArgs a, float* y) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  const long long r = 4 * (blockIdx.x * 8ll + warp);
  if (r >= a.H) return;
  const int p0 = a.first[e], p1 = a.first[e + 1];
  const E* w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = static_cast<const E*>(a.Wd) + (e * a.H + min(r + i, a.H - 1)) * a.I;
  for (int p = p0; p < p1; p += 4) {
    const float* h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = static_cast<const float*>(a.h) + min(p + i, p1 - 1) * a.I;
    float v[16];
    tile16<DT, DETFFN_F32, VEC>(h, w, a.I, lane, v);
    const float s = sum16(v, lane);
    const int of = sum16_of(lane), q = p + (of >> 2);
    const long long c = r + (of & 3);
    if (lane < 16 && q < p1 && c < a.H) y[q * a.H + c] = s;
  }
}

// out of token blockIdx.y: its pairs in the order of its choices.
template <int DT>
__global__ void __launch_bounds__(256) k_combine(const __grid_constant__ MoeArgs a, const float* y) {
  grid_dep_wait();
  grid_dep_launch();
  const int t = blockIdx.y;
  const long long r = blockIdx.x * 256ll + threadIdx.x;
  if (r >= a.H) return;
  float s = 0.0f;
  for (int j = 0; j < a.k; ++j) s = fmaf(a.weights[t * a.k + j], y[a.pos[t * a.k + j] * a.H + r], s);
  Io<DT>::st(static_cast<typename Io<DT>::E*>(a.out) + t * a.H + r, s);
}

template <int DT>
cudaError_t logits(const MoeArgs& a, int* counters, int n, cudaStream_t st) {
  const bool vec = a.H % 8 == 0 && (((uintptr_t)a.x | (uintptr_t)a.Wr) & 15u) == 0;
  if (vec) return launch_dependent(k_logits_tile<DT>, dim3((a.E + 3) / 4, (a.T + 3) / 4), 256, 0, st, a, counters, n);
  return launch_dependent(k_logits<DT>, dim3(a.E), 256, 0, st, a, counters, n);
}

template <int DT>
cudaError_t general(const MoeArgs& a, float* y, cudaStream_t st) {
  const int per = DT == DETFFN_F32 ? 4 : 8;
  auto on16 = [](const void* p) { return ((uintptr_t)p & 15u) == 0; };
  const bool up = a.H % per == 0 && on16(a.x) && on16(a.Wg) && on16(a.Wu), down = a.I % per == 0 && on16(a.Wd);
  cudaError_t e = launch_moe_logits(a, nullptr, 0, st);
  if (e == cudaSuccess) e = launch_dependent(k_select, dim3(1), 1024, 0, st, a);
  if (e == cudaSuccess)
    e = launch_dependent(up ? k_gateup<DT, true> : k_gateup<DT, false>, dim3((unsigned)((a.I + 15) / 16), a.E), 256, 0, st, a);
  if (e == cudaSuccess)
    e = launch_dependent(down ? k_down<DT, true> : k_down<DT, false>, dim3((unsigned)((a.H + 31) / 32), a.E), 256, 0, st, a, y);
  if (e == cudaSuccess)
    e = launch_dependent(k_combine<DT>, dim3((unsigned)((a.H + 255) / 256), a.T), 256, 0, st, a, (const float*)y);
  return e;
}

}  // namespace

cudaError_t launch_moe_logits(const MoeArgs& a, int* counters, int n, cudaStream_t st) {
  return a.dtype == DETFFN_F32 ? logits<DETFFN_F32>(a, counters, n, st)
         : a.dtype == DETFFN_F16 ? logits<DETFFN_F16>(a, counters, n, st) : logits<DETFFN_BF16>(a, counters, n, st);
}

cudaError_t launch_moe_general(const MoeArgs& a, const MoeScratch& sc, cudaStream_t st) {
  return a.dtype == DETFFN_F32 ? general<DETFFN_F32>(a, sc.y, st)
         : a.dtype == DETFFN_F16 ? general<DETFFN_F16>(a, sc.y, st) : general<DETFFN_BF16>(a, sc.y, st);
}

}  // namespace detffn
