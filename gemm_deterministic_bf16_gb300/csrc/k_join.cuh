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
// fixed order, so results do not depend on the run.
#pragma once

#include "block.h"
#include "elt.cuh"

namespace detffn {
namespace join {

// Features c .. c + 7 of a row or a parameter; zeros past the row's end.
template <int DT>
__device__ __forceinline__ void load(const void* base, long long off, int c, int H, float (&v)[8]) {
  using E = typename Io<DT>::E;
  if (c < H) {
    Io<DT>::ld8(static_cast<const E*>(base) + off + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
}
template <int DT>
__device__ __forceinline__ void store(void* base, long long off, int c, int H, const float (&v)[8]) {
  if (c < H) Io<DT>::st8(static_cast<typename Io<DT>::E*>(base) + off + c, v);
}
// A parameter, in the elements' type or in FP32.
template <int DT>
__device__ __forceinline__ void load_param(const void* base, int pdtype, long long off, int c, int H, float (&v)[8]) {
  if (DT == DETFFN_F32 || pdtype == DT) load<DT>(base, off, c, H, v);
  else load<DETFFN_F32>(base, off, c, H, v);
}

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

// A few rows of whole 16-byte vectors and at most 4096 features: one block of
// threads to a row, eight features to a thread, in registers.  Bound by latency,
// so all of a row's loads go out before its sums (one row of 4096 features, BF16:
// 3.1 us).
template <int DT>
__global__ void __launch_bounds__(512) k_fwd(const __grid_constant__ JoinArgs a) {
  __shared__ float buf[2 * 32];
  grid_dep_wait();
  grid_dep_launch();
  const int c = 8 * threadIdx.x, H = a.H;
  const float inv = 1.0f / (float)H;
  int turn = 0;
  auto gate_of = [&](long long m, float (&g)[8]) {
    if (!a.gate) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 1.0f;
    } else if (a.gate_cs) {
      load_param<DT>(a.gate, a.pdtype, m * a.gate_rs, c, H, g);
    } else {
      const float one = param<DT>(a.gate, a.pdtype, m * a.gate_rs);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = one;
    }
  };
  float post[8], pre[8], gate[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) post[j] = pre[j] = 1.0f;
  if (a.w_post) load_param<DT>(a.w_post, a.pdtype, 0, c, H, post);
  if (a.w_pre) load_param<DT>(a.w_pre, a.pdtype, 0, c, H, pre);
  if (!a.gate_rs) gate_of(0, gate);
  for (long long m = blockIdx.x; m < a.M; m += gridDim.x) {
    float r[8], n[8];
    load<DT>(a.x.p, m * a.x.ld, c, H, r);
    if (a.z.p) load<DT>(a.z.p, m * a.z.ld, c, H, n);
    if (a.gate_rs) gate_of(m, gate);
    if (a.z.p) {
      float b = 1.0f;
      if (a.w_post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(n[j], n[j], s[0]);
        block_sums<1>(s, buf, turn);
        b = rsqrtf(s[0] * inv + a.eps);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = fmaf(a.scale, n[j] * (b * post[j]) * gate[j], r[j]);
      store<DT>(const_cast<void*>(a.out.p), m * a.out.ld, c, H, r);
    }
    if (a.w_pre) {
      float s[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(r[j], r[j], s[0]);
      block_sums<1>(s, buf, turn);
      const float q = rsqrtf(s[0] * inv + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] *= q * pre[j];
      store<DT>(const_cast<void*>(a.y.p), m * a.y.ld, c, H, r);
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
