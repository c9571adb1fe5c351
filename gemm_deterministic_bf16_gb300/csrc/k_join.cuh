// k_join.cuh -- the norms before and after a block joined with its gate and
// residual scale: the formulas, the forward kernel for few rows, and the sums
// over row sets (each k_join_*.cu instantiates one element type;
// k_join_ring.cuh has the kernels for the rest).
//
// Forward, for each token (a row of H features):
//   n   = z / sqrt(mean(z^2) + eps) * w_post      (the norm after the block; n = z without w_post)
//   out = x + scale * gate * n
//   y   = out / sqrt(mean(out^2) + eps) * w_pre   (the next block's norm)
// y is formed from the sum before it is rounded to the stored type, so each
// output is rounded once.  Without z, out is x itself and only y is written.
//
// Backward, with a = 1 / sqrt(mean(r^2) + eps), b = 1 / sqrt(mean(z^2) + eps),
// r the stored sum:
//   dx = dr + a dy w_pre - r a^3 / H * sum(dy w_pre r)
//   t  = scale * dx,  dgate = t n,  dn = t gate
//   dz = b dn w_post - z b^3 / H * sum(dn w_post z)
//   dw_pre = sum over tokens of dy r a,  dw_post = sum over tokens of dn z b
// dgate is summed over what the gate is broadcast over (features, tokens or
// both).  Sums over tokens: each block of threads adds the rows of its set
// (rows s, s + sets, ...) in order, and a second kernel adds the sets in a
// fixed order, so results do not depend on the run.  What a set is depends on the
// sizes, the types, the norms and gate there are and the alignment; a row's own
// results depend on H, the types and the alignment.
#pragma once

#include "block.h"
#include "elt.cuh"

namespace detffn {
namespace join {

template <int DT>
__device__ __forceinline__ float param(const void* base, int pdtype, long long i) {
  if (DT == DETFFN_F32 || pdtype == DT) return Io<DT>::ld(static_cast<const typename Io<DT>::E*>(base) + i);
  return static_cast<const float*>(base)[i];
}
template <int DT>
__device__ __forceinline__ void put_param(void* base, int pdtype, long long i, float v) {
  if (DT == DETFFN_F32 || pdtype == DT) Io<DT>::st(static_cast<typename Io<DT>::E*>(base) + i, v);
  else static_cast<float*>(base)[i] = v;
}

// Sums of N = 2 or 4 values over a group of G threads (whole warps, at most
// 20), the same in every thread, in an order fixed by G.  Stage one halves the
// values a lane carries with every exchange, so that lane l ends with the
// warp's sum of value l % N; stage two adds the warps the same way, through
// [2][20 N] floats.  One barrier; one warp alone: none but __syncwarp.
template <int N, int THREADS = 512>
struct GroupSums {
  static_assert(N == 2 || N == 4, "");
  float *put, *get;     // this thread's places, now in the first half
  int other = 20 * N;   // the other half, from there
  int warps, barrier, threads;
  bool odd, high;
  // `buf`: 40 N floats of the group.
  __device__ __forceinline__ GroupSums(float* buf, int G, int group, int t) {
    const int lane = t & 31;
    put = buf + (t >> 5) * N + lane;
    get = buf + lane;
    warps = (G >> 5) * N - lane;   // 0 or less: no value for this lane
    barrier = group + 1;
    threads = G;
    odd = lane & 1;
    high = lane & 2;
  }
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    float x = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
    if (N == 4) {
      const float c = v[N - 2], d = v[N - 1];
      const float y = (odd ? d : c) + __shfl_xor_sync(0xffffffffu, odd ? c : d, 1);
      x = (high ? y : x) + __shfl_xor_sync(0xffffffffu, high ? x : y, 2);
    }
#pragma unroll
    for (int s = N; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    if (threads > 32) {
      if ((int)(threadIdx.x & 31) < N) *put = x;
      asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
      x = warps > 0 ? get[0] : 0.0f;
      if (N == 4) x += warps > 32 ? get[32] : 0.0f;
      if (N == 4 && THREADS > 512) x += warps > 64 ? get[64] : 0.0f;
      put += other;
      get += other;
      other = -other;
#pragma unroll
      for (int s = N; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    } else {
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x, i);
  }
};

// One unit of a thread: with VEC features c .. c + 7 (a thread past the row's
// end reads the last unit and counts for nothing: on is 0), else c + 32 j where
// bit j of on is set, and zeros.
struct Cols {
  int c;
  uint32_t on;
};
template <bool VEC>
__device__ __forceinline__ Cols cols_of(int i, int G, int t, int H) {
  Cols k;
  if (VEC) {
    k.on = 8 * (i * G + t) < H;
    k.c = k.on ? 8 * (i * G + t) : H - 8;
  } else {
    k.c = 256 * (i * (G >> 5) + (t >> 5)) + (t & 31);
    k.on = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) k.on |= (k.c + 32 * j < H ? 1u : 0u) << j;
  }
  return k;
}
template <int DT, bool VEC>
__device__ __forceinline__ void unit(const void* row, const Cols& k, float (&v)[8]) {
  using E = typename Io<DT>::E;
  const E* p = static_cast<const E*>(row) + k.c;
  if (VEC) {
    Io<DT>::ld8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k.on >> j & 1 ? Io<DT>::ld(p + 32 * j) : 0.0f;
  }
}
template <int DT, bool VEC>
__device__ __forceinline__ void put_unit(void* row, const Cols& k, const float (&v)[8]) {
  using E = typename Io<DT>::E;
  E* p = static_cast<E*>(row) + k.c;
  if (VEC) {
    if (k.on) Io<DT>::st8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k.on >> j & 1) Io<DT>::st(p + 32 * j, v[j]);
  }
}
// The same of a parameter, in the rows' type or FP32; `fill` where there is none.
template <int DT, bool VEC>
__device__ __forceinline__ void param_unit(const void* p, int pdtype, const Cols& k, float fill, float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fill;
  } else if (DT == DETFFN_F32 || pdtype == DT) {
    unit<DT, VEC>(p, k, v);
  } else {
    unit<DETFFN_F32, VEC>(p, k, v);
  }
}
__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
  float s = a[0] * b[0], q = a[1] * b[1];
#pragma unroll
  for (int j = 2; j < 8; j += 2) s = fmaf(a[j], b[j], s), q = fmaf(a[j + 1], b[j + 1], q);
  return s + q;
}

// Sum over a block of at most 16 warps, the same in every thread: a tree over the
// lanes, then over the warps, neighbours first -- as GroupSums adds one value.
// `buf`: [2][16] floats; one barrier, as its halves take turns.
__device__ __forceinline__ float tree_sum(float x, float* buf, int& turn) {
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  if (warps == 1) return x;
  float* b = buf + turn * 16;
  turn ^= 1;
  if (lane == 0) b[threadIdx.x >> 5] = x;
  __syncthreads();
  x = lane < warps ? b[lane] : 0.0f;
#pragma unroll
  for (int s = 1; s < 16; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return __shfl_sync(0xffffffffu, x, 0);
}

// A few rows of whole 16-byte vectors and at most 4096 features: one block of
// threads to a row, a unit to a thread, in registers.  Every sum and product is
// the ring kernel's, in its order, so that a row's bits do not depend on how many
// rows the call has: where a thread there holds units t and G + t, neighbours
// hold them here (PAIR), and their sum is the first of the tree.  Bound by
// latency, so all of a row's loads go out before its sums (one row of 4096
// features, BF16: 2.9 us; with two units to a thread, 3.5).
template <int DT, bool PAIR>
__global__ void __launch_bounds__(512) k_fwd(const __grid_constant__ JoinArgs a) {
  __shared__ float buf[2 * 16];
  grid_dep_wait();
  grid_dep_launch();
  const int H = a.H, t = threadIdx.x;
  const float inv = 1.0f / (float)H;
  const bool by_row = a.gate && a.gate_rs;
  int turn = 0;
  const Cols k = cols_of<true>(0, 0, PAIR ? (t >> 1) + (t & 1) * (int)(blockDim.x >> 1) : t, H);
  float mix[8], pre[8];      // mix: scale * gate * w_post
  {
    float w[8];
    param_unit<DT, true>(a.w_pre, a.pdtype, k, 1.0f, pre);
    param_unit<DT, true>(a.w_post, a.pdtype, k, 1.0f, w);
    param_unit<DT, true>(a.gate_cs && !by_row ? a.gate : nullptr, a.pdtype, k,
                         a.gate && !a.gate_cs && !by_row ? param<DT>(a.gate, a.pdtype, 0) : 1.0f, mix);
#pragma unroll
    for (int j = 0; j < 8; ++j) mix[j] *= a.scale * w[j];
  }
  for (long long m = blockIdx.x; m < a.M; m += gridDim.x) {
    auto row = [&](const Rows& r) { return static_cast<const typename Io<DT>::E*>(r.p) + m * r.ld; };
    float r[8], z[8], g[8];
    unit<DT, true>(row(a.x), k, r);
    if (a.z.p) unit<DT, true>(row(a.z), k, z);
    if (by_row) {
      const char* gate = static_cast<const char*>(a.gate) + m * a.gate_rs * (a.pdtype == DETFFN_F32 ? 4 : 2);
      param_unit<DT, true>(a.gate_cs ? gate : nullptr, a.pdtype, k, a.gate_cs ? 0.0f : param<DT>(gate, a.pdtype, 0), g);
    }
    if (a.z.p) {
      float b = 1.0f;
      if (a.w_post) b = rsqrtf(fmaf(tree_sum(k.on ? dot8(z, z) : 0.0f, buf, turn), inv, a.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = fmaf(b * z[j], by_row ? g[j] * mix[j] : mix[j], r[j]);
      put_unit<DT, true>(const_cast<typename Io<DT>::E*>(row(a.out)), k, r);
    }
    if (a.w_pre) {
      const float q = rsqrtf(fmaf(tree_sum(k.on ? dot8(r, r) : 0.0f, buf, turn), inv, a.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] *= q * pre[j];
      put_unit<DT, true>(const_cast<typename Io<DT>::E*>(row(a.y)), k, r);
    }
  }
}

constexpr int kSetReads = 10;   // (152 sets in 16 runs)

// out[c] = sum over sets of part[s][c]: Q = blockDim / 32 threads per column
// take sets q, q + Q, ... in order and their sums are added in order.  Bound by
// latency, so a thread's reads are all under way at once.
template <int DT>
__global__ void __launch_bounds__(512) k_sets(const float* __restrict__ part, int sets, long long n, void* out0,
                                              void* out1, void* out2, long long per, int pdtype) {
  __shared__ float s[16][33];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5, Q = blockDim.x >> 5;
  const long long c = blockIdx.x * 32ll + lane;
  const float* p = part + blockIdx.y * per + c;
  float v = 0.0f;
  if (c < n) {
#pragma unroll
    for (int k = 0; k < kSetReads; ++k)   // (all reads under way before the first addition)
      if (q + k * Q < sets) v += __ldcg(p + (long long)(q + k * Q) * n);
  }
  s[q][lane] = v;
  __syncthreads();
  if (q == 0 && c < n) {
    for (int k = 1; k < Q; ++k) v += s[k][lane];
    put_param<DT>(blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2, pdtype, c, v);
  }
}
static_assert(kJoinSets <= 16 * kSetReads, "a thread of k_sets reads at most kSetReads sets");
inline int sets_threads(int sets) { return sets <= 8 * kSetReads ? 256 : 512; }

inline bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Whether every row access of the call is whole 16-byte vectors.
template <int DT>
bool vectors(const JoinArgs& a) {
  if (a.H % 8) return false;
  const Rows* rows[] = {&a.x, &a.z, &a.out, &a.y, &a.r, &a.dr, &a.dy, &a.dx, &a.dz};
  for (const Rows* r : rows)
    if (r->p && (!on16(r->p) || (r->ld * Io<DT>::kBytes) % 16)) return false;
  const int pb = a.pdtype == DETFFN_F32 ? 4 : 2;
  if (!on16(a.w_post) || !on16(a.w_pre)) return false;
  if (a.gate && a.gate_cs && (!on16(a.gate) || (a.gate_rs * pb) % 16 || !on16(a.dgate))) return false;
  return true;
}

}  // namespace join
}  // namespace detffn
