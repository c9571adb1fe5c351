// k_ckpt.cu -- activation checkpoints in 8 bits: gate and up written as signed
// 8-bit codes with one FP32 scale per 64 consecutive features of a token, read
// back, and used by the SiLU stage of the backward pass.
//
//   s = max|v| / 127 over the block,  q = rint(v / s) in [-127, 127]
//   value = q * s
//
// A block of zeros has s = 0 and q = 0.  A block that holds an infinity or a
// NaN has s = NaN: all its values read back as NaN, so that an overflow shows
// in the gradients instead of being clipped.
//
// The backward stage works from the stored values in FP32 and rounds each of
// its three outputs once:
//   sigma = 1 / (1 + exp(-g)), a = g sigma
//   dU = dh a,  dG = dh u sigma (1 + g (1 - sigma)),  h = a u
#include "block.h"
#include "elt.cuh"

namespace detffn {
namespace {

constexpr int kThreads = 256;
constexpr float kInv127 = 1.0f / 127.0f;
constexpr float kTopScale = 0x1.0204060000000p+121f;  // the largest scale whose 127-fold is finite

// The code of v at scale s: rint of the correctly rounded quotient.
__device__ __forceinline__ int code_of(float v, float s) {
  const float q = rintf(__fdiv_rn(v, s));
  return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

__device__ __forceinline__ float scale_of(float top, bool finite) {
  return finite ? fminf(__fmul_rn(top, kInv127), kTopScale) : __int_as_float(0x7fc00000);
}

// Eight lanes take one block of 64 features; lane l holds features l, l + 8,
// ... (any row length) or 8 l .. 8 l + 7 (rows of whole 16-byte vectors).
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_pack(CkptArgs a, long long nb) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int l = threadIdx.x & 7;
  const long long groups = (long long)gridDim.x * (kThreads / 8), total = 2 * a.M * nb;
  // Whole warps stay in the loop: the shuffles below need all their lanes.
  for (long long t0 = (blockIdx.x * (long long)kThreads + (threadIdx.x & ~31)) / 8; t0 < total; t0 += groups) {
    const long long t = t0 + ((threadIdx.x & 31) >> 3);
    const bool on = t < total;
    const long long u = on ? t : total - 1;
    const bool second = u >= a.M * nb;
    const long long b = second ? u - a.M * nb : u;
    const long long m = b / nb, c0 = (b - m * nb) * kCkptBlock;
    const E* src = static_cast<const E*>(second ? a.up : a.gate) + m * a.I + c0;
    int8_t* dst = (second ? a.uq : a.gq) + m * a.I + c0;
    const int n = (int)(a.I - c0 < kCkptBlock ? a.I - c0 : kCkptBlock);
    float v[8];
    if (VEC) {
      if (8 * l < n) Io<DT>::ld8(src + 8 * l, v);
      else
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = l + 8 * j < n ? Io<DT>::ld(src + l + 8 * j) : 0.0f;
    }
    float top = 0.0f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      finite = finite && fabsf(v[j]) <= 3.402823466e38f;
      top = fmaxf(top, fabsf(v[j]));
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      finite = __shfl_xor_sync(0xffffffffu, (int)finite, d) && finite;
    }
    const float s = scale_of(top, finite);
    if (!on) continue;
    if (l == 0) (second ? a.us : a.gs)[b] = s;
    int q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = s > 0.0f ? code_of(v[j], s) : 0;
    if (VEC) {
      if (8 * l < n) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo |= (uint32_t)(q[j] & 255) << (8 * j);
          hi |= (uint32_t)(q[4 + j] & 255) << (8 * j);
        }
        *reinterpret_cast<uint2*>(dst + 8 * l) = make_uint2(lo, hi);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (l + 8 * j < n) dst[l + 8 * j] = (int8_t)q[j];
    }
  }
}

// Eight codes as values.
__device__ __forceinline__ void values8(uint2 q, float s, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = __fmul_rn((float)(int8_t)(q.x >> (8 * j)), s);
    v[4 + j] = __fmul_rn((float)(int8_t)(q.y >> (8 * j)), s);
  }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_unpack(CkptArgs a, long long nb) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  constexpr int PER = VEC ? 8 : 1;
  const long long per_row = a.I / PER, half = a.M * per_row;
  for (long long t = blockIdx.x * (long long)kThreads + threadIdx.x; t < 2 * half;
       t += (long long)gridDim.x * kThreads) {
    const bool second = t >= half;
    const long long i = second ? t - half : t, m = i / per_row, c = (i - m * per_row) * PER, at = m * a.I + c;
    const float s = (second ? a.us : a.gs)[m * nb + c / kCkptBlock];
    const int8_t* q = (second ? a.uq : a.gq) + at;
    E* dst = static_cast<E*>(const_cast<void*>(second ? a.up : a.gate)) + at;
    if (VEC) {
      float v[8];
      values8(*reinterpret_cast<const uint2*>(q), s, v);
      Io<DT>::st8(dst, v);
    } else {
      Io<DT>::st(dst, __fmul_rn((float)*q, s));
    }
  }
}

__device__ __forceinline__ void silu_stage(float dh, float g, float u, float& dU, float& dG, float& h) {
  const float sig = __fdividef(1.0f, 1.0f + __expf(-g));
  const float act = g * sig;
  dU = dh * act;
  dG = dh * u * (sig * (1.0f + g * (1.0f - sig)));
  h = act * u;
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_bwd(CkptArgs a, long long nb) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  constexpr int PER = VEC ? 8 : 1;
  const long long per_row = a.I / PER, total = a.M * per_row;
  const E* dh = static_cast<const E*>(a.dh);
  E *oU = static_cast<E*>(a.dU), *oG = static_cast<E*>(a.dG), *oh = static_cast<E*>(a.h);
  for (long long t = blockIdx.x * (long long)kThreads + threadIdx.x; t < total;
       t += (long long)gridDim.x * kThreads) {
    const long long m = t / per_row, c = (t - m * per_row) * PER, at = m * a.I + c, b = m * nb + c / kCkptBlock;
    const float sg = a.gs[b], su = a.us[b];
    if (VEC) {
      float d[8], g[8], u[8], vU[8], vG[8], vh[8];
      Io<DT>::ld8(dh + at, d);
      values8(*reinterpret_cast<const uint2*>(a.gq + at), sg, g);
      values8(*reinterpret_cast<const uint2*>(a.uq + at), su, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) silu_stage(d[j], g[j], u[j], vU[j], vG[j], vh[j]);
      Io<DT>::st8(oU + at, vU);
      Io<DT>::st8(oG + at, vG);
      if (oh) Io<DT>::st8(oh + at, vh);
    } else {
      float vU, vG, vh;
      silu_stage(Io<DT>::ld(dh + at), __fmul_rn((float)a.gq[at], sg), __fmul_rn((float)a.uq[at], su), vU, vG, vh);
      Io<DT>::st(oU + at, vU);
      Io<DT>::st(oG + at, vG);
      if (oh) Io<DT>::st(oh + at, vh);
    }
  }
}

bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool on8(const void* p) { return ((uintptr_t)p & 7u) == 0; }

int grid_for(long long threads, int sm_count) {
  const long long want = (threads + kThreads - 1) / kThreads, most = (long long)sm_count * 8;
  return (int)(want < most ? want : most);
}

template <int DT>
cudaError_t pack(const CkptArgs& a, int sms, cudaStream_t st) {
  const long long nb = (a.I + kCkptBlock - 1) / kCkptBlock;
  const bool vec = a.I % 8 == 0 && on16(a.gate) && on16(a.up) && on8(a.gq) && on8(a.uq);
  return launch_dependent(vec ? k_pack<DT, true> : k_pack<DT, false>, dim3(grid_for(2 * a.M * nb * 8, sms)), kThreads,
                          0, st, a, nb);
}
template <int DT>
cudaError_t unpack(const CkptArgs& a, int sms, cudaStream_t st) {
  const long long nb = (a.I + kCkptBlock - 1) / kCkptBlock;
  const bool vec = a.I % 8 == 0 && on16(a.gate) && on16(a.up) && on8(a.gq) && on8(a.uq);
  return launch_dependent(vec ? k_unpack<DT, true> : k_unpack<DT, false>,
                          dim3(grid_for(2 * a.M * (vec ? a.I / 8 : a.I), sms)), kThreads, 0, st, a, nb);
}
template <int DT>
cudaError_t bwd(const CkptArgs& a, int sms, cudaStream_t st) {
  const long long nb = (a.I + kCkptBlock - 1) / kCkptBlock;
  const bool vec = a.I % 8 == 0 && on16(a.dh) && on16(a.dU) && on16(a.dG) && on16(a.h) && on8(a.gq) && on8(a.uq);
  return launch_dependent(vec ? k_bwd<DT, true> : k_bwd<DT, false>, dim3(grid_for(a.M * (vec ? a.I / 8 : a.I), sms)),
                          kThreads, 0, st, a, nb);
}

}  // namespace

cudaError_t launch_ckpt8_pack(const CkptArgs& a, int sms, cudaStream_t st) {
  return a.dtype == DETFFN_F32 ? pack<DETFFN_F32>(a, sms, st)
         : a.dtype == DETFFN_F16 ? pack<DETFFN_F16>(a, sms, st) : pack<DETFFN_BF16>(a, sms, st);
}
cudaError_t launch_ckpt8_unpack(const CkptArgs& a, int sms, cudaStream_t st) {
  return a.dtype == DETFFN_F32 ? unpack<DETFFN_F32>(a, sms, st)
         : a.dtype == DETFFN_F16 ? unpack<DETFFN_F16>(a, sms, st) : unpack<DETFFN_BF16>(a, sms, st);
}
cudaError_t launch_ckpt8_silu_bwd(const CkptArgs& a, int sms, cudaStream_t st) {
  return a.dtype == DETFFN_F32 ? bwd<DETFFN_F32>(a, sms, st)
         : a.dtype == DETFFN_F16 ? bwd<DETFFN_F16>(a, sms, st) : bwd<DETFFN_BF16>(a, sms, st);
}

}  // namespace detffn
