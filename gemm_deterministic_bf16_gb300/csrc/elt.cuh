// elt.cuh -- reading and writing FP32, FP16 and BF16 elements as FP32 values,
// one at a time or eight at once, and sums over a warp.
#pragma once

#include "common.cuh"

namespace detffn {

// Storage of one element type (a detffn_dtype).  ld8/st8 move eight
// consecutive elements whose address is 16-byte aligned.
template <int DT> struct Io;

template <> struct Io<DETFFN_F32> {
  using E = float;
  static constexpr int kBytes = 4;
  __device__ static float ld(const E* p) { return *p; }
  __device__ static void st(E* p, float v) { *p = v; }
  __device__ static void ld8(const E* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ static void st8(E* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <> struct Io<DETFFN_F16> {
  using E = uint16_t;
  static constexpr int kBytes = 2;
  __device__ static float ld(const E* p) { return __half2float(__ushort_as_half(*p)); }
  __device__ static void st(E* p, float v) { *p = __half_as_ushort(__float2half_rn(v)); }
  __device__ static float round(float v) { return __half2float(__float2half_rn(v)); }
  __device__ static float2 two(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  __device__ static uint32_t pair(float lo, float hi) { return pack_f16x2(lo, hi); }
  __device__ static void ld8(const E* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const float2 a = two(q.x), b = two(q.y), c = two(q.z), d = two(q.w);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
  }
  __device__ static void st8(E* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7]));
  }
};

template <> struct Io<DETFFN_BF16> {
  using E = uint16_t;
  static constexpr int kBytes = 2;
  __device__ static float ld(const E* p) { return bf2f(*p); }
  __device__ static void st(E* p, float v) { *p = f2bf(v); }
  __device__ static float round(float v) { return bf2f(f2bf(v)); }
  __device__ static float2 two(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ static uint32_t pair(float lo, float hi) { return pack_bf16_pair(lo, hi); }
  __device__ static void ld8(const E* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const float2 a = two(q.x), b = two(q.y), c = two(q.z), d = two(q.w);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
  }
  __device__ static void st8(E* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7]));
  }
};

// sigma(g) = 1 / (1 + exp(-g)) and 1 - sigma(g), from exp(-|g|) so that nothing
// overflows and neither loses digits to a subtraction.  FAST: by __expf and
// __fdividef, whose error is about (1.2 |g| + 4) 2^-23 of either (2^-16 at the
// most, where exp leaves the type's range): for results of 16 bits.
struct Sigma {
  float s, rest;
};
template <bool FAST>
__device__ __forceinline__ Sigma sigma(float g) {
  const float e = FAST ? __expf(-fabsf(g)) : expf(-fabsf(g));
  const float big = FAST ? __fdividef(1.0f, 1.0f + e) : 1.0f / (1.0f + e), small = e * big;
  return g < 0.0f ? Sigma{small, big} : Sigma{big, small};
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

}  // namespace detffn
