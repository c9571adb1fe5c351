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
//   sigma = 1 / (1 + exp(-g)) (elt.cuh), a = g sigma
//   dU = dh a,  dG = dh u sigma (1 + g (1 - sigma)),  h = a u
//
// All of it is bound by HBM where vectors carry it: 4096 x 12288 BF16 packs in
// 49.6 us (93 % of the copy rate), unpacks in 46.5 (99 %), and the backward stage
// takes 75 to 76 (100 %).
#include <type_traits>

#include "block.h"
#include "elt.cuh"

namespace detffn {
namespace {

constexpr int kThreads = 256;
constexpr float kInv127 = 1.0f / 127.0f;
constexpr float kTopScale = 0x1.0204060000000p+121f;  // the largest scale whose 127-fold is finite
constexpr float kMagic = 12582912.0f;                 // 1.5 2^23: v + kMagic rounds |v| < 2^22 to a whole number

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994).
struct Div {
  uint32_t mul = 0, shift = 0, d = 1;
};
Div div_by(uint32_t d) {
  Div r;
  r.d = d;
  while ((1ull << r.shift) < d) ++r.shift;
  r.mul = (uint32_t)(((1ull << 32) * ((1ull << r.shift) - d)) / d + 1);
  return r;
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Div& v) { return (__umulhi(n, v.mul) + n) >> v.shift; }

// Bits of |v|: as whole numbers these are in the order of the values, with the
// infinities and NaNs above all numbers.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Codes of N values at scale s > 0, each in a word's low byte: rint of the
// correctly rounded quotient.  One correction of v * (1 / s) by its exact
// remainder gives that (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990); scales so small that a step could
// underflow divide instead.
constexpr float kPlainScale = 1e-30f;
__device__ __forceinline__ uint32_t code_at(float v, float s, float inv) {   // (s >= kPlainScale)
  const float t = v * inv;
  return __float_as_uint(fmaf(fmaf(-t, s, v), inv, t) + kMagic);
}
template <int N>
__device__ __forceinline__ void code_bits(const float (&v)[N], float s, uint32_t (&q)[N]) {
  const float inv = __fdividef(1.0f, s);
#pragma unroll
  for (int j = 0; j < N; ++j) q[j] = code_at(v[j], s, inv);
  if (s < kPlainScale) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      q[j] = __float_as_uint(fminf(fmaxf(rintf(__fdiv_rn(v[j], s)), -127.0f), 127.0f) + kMagic);
  }
}

// Four codes in a word.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Four codes as values: a byte under the exponent of 2^23 is 2^23 + 128 more
// than the code, so one exact subtraction converts it.
__device__ __forceinline__ float code_value(uint32_t w, int j) {  // (w: the codes ^ 0x80)
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + j)) - 8388736.0f;
}

// N = 16 bytes' worth of consecutive elements: eight of 16 bits, four of 32.
template <int DT> constexpr int kPer = DT == DETFFN_F32 ? 4 : 8;
template <int DT>
__device__ __forceinline__ void load_vec(const typename Io<DT>::E* p, float (&v)[kPer<DT>]) {
  if constexpr (DT == DETFFN_F32) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
    Io<DT>::ld8(p, v);
  }
}
template <int DT>
__device__ __forceinline__ void store_vec(typename Io<DT>::E* p, const float (&v)[kPer<DT>]) {
  if constexpr (DT == DETFFN_F32) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else Io<DT>::st8(p, v);
}
// Their codes, as the words they fill.
template <int DT>
__device__ __forceinline__ void load_codes(const int8_t* p, uint32_t (&w)[kPer<DT> / 4]) {
  if constexpr (DT == DETFFN_F32) {
    w[0] = *reinterpret_cast<const uint32_t*>(p) ^ 0x80808080u;
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    w[0] = q.x ^ 0x80808080u, w[1] = q.y ^ 0x80808080u;
  }
}

__device__ __forceinline__ float scale_of(uint32_t top) {
  return top < 0x7F800000u ? fminf(__fmul_rn(__uint_as_float(top), kInv127), kTopScale) : __int_as_float(0x7fc00000);
}

// Rows of whole 8-element vectors on 16-byte boundaries: four lanes take one
// block of 64 features, of gate and of up, lane l features 8 l .. 8 l + 7 and
// 32 more than those: four loads under way, and three exchanges for 32 values
// (56 us at 4096 x 12288 BF16 with eight lanes and half of both, 49.6 so).
// FLAT: no block is short (I a multiple of 64), so blocks follow one another and
// nothing is divided.
template <int DT, bool FLAT>
__global__ void __launch_bounds__(kThreads) k_pack_vec(const __grid_constant__ CkptArgs a, uint32_t blocks, Div nb) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int l = threadIdx.x & 3;
  const uint32_t step = gridDim.x * (kThreads / 4);
  // Whole warps stay in the loop: the shuffles need all their lanes.
  for (uint32_t b0 = (blockIdx.x * kThreads + (threadIdx.x & ~31u)) / 4; b0 < blocks; b0 += step) {
    const uint32_t b = min(b0 + ((threadIdx.x & 31) >> 2), blocks - 1);   // (past the last: the last again)
    long long at = 64ll * b + 8 * l;
    bool on[2] = {true, true};
    if (!FLAT) {
      const uint32_t m = quotient(b, nb), c = (b - m * nb.d) * kCkptBlock + 8 * l;
      at = (long long)m * a.I + c;
      on[0] = c < a.I;
      on[1] = c + 32 < a.I;
    }
    // Values 2 k + i: vector i of gate (k = 0) or up (1).
    float v[4][8];
    uint32_t top[2] = {0, 0};
    if constexpr (DT == DETFFN_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const E* p = static_cast<const E*>(i >> 1 ? a.up : a.gate) + at + 32 * (i & 1);
        if (on[i & 1]) {
          Io<DT>::ld8(p, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) top[i >> 1] = max(top[i >> 1], mag_bits(v[i][j]));
    } else {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const E* p = static_cast<const E*>(i >> 1 ? a.up : a.gate) + at + 32 * (i & 1);
        q[i] = on[i & 1] ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
      }
      // The largest of 16-bit magnitudes, two to an instruction.
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = Io<DT>::two(w[j]);
          v[i][2 * j] = f.x;
          v[i][2 * j + 1] = f.y;
          top[i >> 1] = __vmaxu2(top[i >> 1], w[j] & 0x7FFF7FFFu);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) top[k] = mag_bits(Io<DT>::two(max(top[k] & 0xFFFFu, top[k] >> 16)).x);
    }
    // Gate's and up's largest in one exchange less: lane bit 0 keeps one each.
    {
      const bool up = l & 1;
      uint32_t t = max(up ? top[1] : top[0], __shfl_xor_sync(0xffffffffu, up ? top[0] : top[1], 1));
      t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
      const uint32_t o = __shfl_xor_sync(0xffffffffu, t, 1);
      top[0] = up ? o : t;
      top[1] = up ? t : o;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float s = scale_of(top[k]);
      if (l == 0) (k ? a.us : a.gs)[b] = s;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint2 w = make_uint2(0, 0);
        if (s > 0.0f) {
          uint32_t q[8];
          code_bits(v[2 * k + i], s, q);
          w = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
        }
        if (on[i]) *reinterpret_cast<uint2*>((k ? a.uq : a.gq) + at + 32 * i) = w;
      }
    }
  }
}

// Any row length and alignment: a warp takes four blocks, a lane features
// lane and lane + 32 of each (64 bytes of a row to an access), of gate and up.
// Bound by issue, as every element is loaded, coded and stored by itself; four
// whole blocks of one row, which most are, share an address and need no tests
// (4096 x 12283 BF16: 109 us without that case, 77 so, 60 % of the copy
// rate; aligned vectors whose blocks' maxima meet in shared memory by atomics
// took 121).
template <int DT>
__global__ void __launch_bounds__(kThreads) k_pack_any(const __grid_constant__ CkptArgs a, uint32_t blocks, Div nb) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  const int lane = threadIdx.x & 31;
  const uint32_t step = gridDim.x * (kThreads / 32) * 4;
  for (uint32_t b0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * 4; b0 < blocks; b0 += step) {
    const uint32_t m0 = quotient(b0, nb), c0 = (b0 - m0 * nb.d) * kCkptBlock;
    const long long at0 = (long long)m0 * a.I + c0 + lane;
    auto four = [&](const bool whole) __attribute__((always_inline)) {
      long long at[4];
      int n[4];
      float v[8][2];     // value 2 i + k: block i of gate (0) or up (1)
      uint32_t top[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (whole) {
          at[i] = at0 + 64 * i;
          n[i] = 64;
        } else {
          const uint32_t b = min(b0 + i, blocks - 1), m = quotient(b, nb), c = (b - m * nb.d) * kCkptBlock;
          at[i] = (long long)m * a.I + c + lane;
          n[i] = (int)min(a.I - c, (long long)kCkptBlock) - lane;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const E* p = static_cast<const E*>(k ? a.up : a.gate) + at[i];
          v[2 * i + k][0] = n[i] > 0 ? Io<DT>::ld(p) : 0.0f;
          v[2 * i + k][1] = n[i] > 32 ? Io<DT>::ld(p + 32) : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = max(mag_bits(v[i][0]), mag_bits(v[i][1]));
      // Lane l ends with the largest of value l & 7 (each exchange halves what a
      // lane carries), and every lane then fetches all eight.
#pragma unroll
      for (int d = 0; d < 3; ++d) {
        const bool up = lane >> d & 1;
#pragma unroll
        for (int i = 0; i < 4 >> d; ++i) {
          const uint32_t lo = top[2 * i], hi = top[2 * i + 1];
          top[i] = max(up ? hi : lo, __shfl_xor_sync(0xffffffffu, up ? lo : hi, 1 << d));
        }
      }
      top[0] = max(top[0], __shfl_xor_sync(0xffffffffu, top[0], 8));
      top[0] = max(top[0], __shfl_xor_sync(0xffffffffu, top[0], 16));
      const float mine = scale_of(top[0]);
      if (lane < 8 && (whole || b0 + (lane >> 1) < blocks)) (lane & 1 ? a.us : a.gs)[b0 + (lane >> 1)] = mine;
      const float inv = __fdividef(1.0f, mine);
      const bool plain = __all_sync(0xffffffffu, mine >= kPlainScale);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = __shfl_sync(0xffffffffu, mine, i), r = __shfl_sync(0xffffffffu, inv, i);
        uint32_t q[2] = {code_at(v[i][0], s, r), code_at(v[i][1], s, r)};
        if (!plain) {   // (a scale is 0, NaN or tiny)
          q[0] = q[1] = 0;
          if (s > 0.0f) code_bits(v[i], s, q);
        }
        int8_t* p = (i & 1 ? a.uq : a.gq) + at[i >> 1];
        if (n[i >> 1] > 0) p[0] = (int8_t)q[0];
        if (n[i >> 1] > 32) p[32] = (int8_t)q[1];
      }
    };
    if (c0 + 4 * kCkptBlock <= a.I) four(true);
    else four(false);
  }
}

// How the kernels that read a checkpoint take its elements.
//   kFlat: 16-byte vectors, I a multiple of 64: a vector's scale is that of its
//          position in the whole tensor;
//   kRows: vectors that no block's end divides (I a multiple of the vector);
//   kMixed: vectors of the tensor as one array, whatever I >= 8 is: up to three
//          blocks meet in one (a block's end, a short block, a row's end);
//   kOne:  element by element.
// kMixed costs selects: 4096 x 12283 BF16 unpacks in 62.5 us (74 % of the copy
// rate, kFlat 99 %), and its backward stage takes 102 (75 %, kFlat 100 %).
enum Mode { kFlat, kRows, kMixed, kOne };

// The scales of one vector: element j has s[0] for j < e0, s[1] for j < e1,
// then s[2].
struct Scales {
  float s[3];
  int e0, e1;
  __device__ __forceinline__ float of(int j) const { return j < e0 ? s[0] : j < e1 ? s[1] : s[2]; }
};
template <int PER, Mode MODE>
__device__ __forceinline__ Scales scales_at(const float* s, long long block, uint32_t c, long long I, long long blocks) {
  Scales r;
  r.s[0] = s[block];
  r.e0 = r.e1 = PER;
  if (MODE == kMixed) {
    const int left = (int)min((long long)(kCkptBlock - c % kCkptBlock), I - c);
    r.s[1] = r.s[2] = r.s[0];
    if (left < PER) {
      r.e0 = left;
      r.s[1] = s[min(block + 1, blocks - 1)];
      // The next block is short only at a row's end.
      const long long next = c + left == I ? 0 : c + left;
      r.e1 = left + (int)min((long long)kCkptBlock, I - next);
      if (r.e1 < PER) r.s[2] = s[min(block + 2, blocks - 1)];
    }
  }
  return r;
}

template <int DT, Mode MODE>
__global__ void __launch_bounds__(kThreads) k_unpack(const __grid_constant__ CkptArgs a, uint32_t n, Div row, int nb) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  constexpr int PER = MODE == kOne ? 1 : kPer<DT>;
  const long long blocks = a.M * nb, total = a.M * a.I;
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) {
    const long long at = (long long)i * PER;
    uint32_t c = 0;
    long long b = at / kCkptBlock;
    if (MODE != kFlat) {
      const uint32_t m = quotient(i * PER, row);
      c = i * PER - m * row.d;
      b = (long long)m * nb + c / kCkptBlock;
    }
    E *g = static_cast<E*>(const_cast<void*>(a.gate)) + at, *u = static_cast<E*>(const_cast<void*>(a.up)) + at;
    if constexpr (MODE == kOne) {
      Io<DT>::st(g, __fmul_rn((float)a.gq[at], a.gs[b]));
      Io<DT>::st(u, __fmul_rn((float)a.uq[at], a.us[b]));
    } else {
      const Scales sg = scales_at<PER, MODE>(a.gs, b, c, a.I, blocks), su = scales_at<PER, MODE>(a.us, b, c, a.I, blocks);
      if (MODE == kMixed && at + PER > total) {   // the array's last elements
        for (int j = 0; at + j < total; ++j) {
          Io<DT>::st(g + j, __fmul_rn((float)a.gq[at + j], sg.of(j)));
          Io<DT>::st(u + j, __fmul_rn((float)a.uq[at + j], su.of(j)));
        }
        continue;
      }
      uint32_t qg[PER / 4], qu[PER / 4];
      load_codes<DT>(a.gq + at, qg);
      load_codes<DT>(a.uq + at, qu);
      float v[PER], w[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        v[j] = code_value(qg[j / 4], j % 4) * sg.of(j);
        w[j] = code_value(qu[j / 4], j % 4) * su.of(j);
      }
      store_vec<DT>(g, v);
      store_vec<DT>(u, w);
    }
  }
}

template <int DT>
__device__ __forceinline__ void silu_stage(float dh, float g, float u, float& dU, float& dG, float& h) {
  const Sigma sig = sigma<DT != DETFFN_F32>(g);
  const float act = g * sig.s;
  dU = dh * act;
  dG = dh * u * (sig.s * (1.0f + g * sig.rest));
  h = act * u;
}

template <int DT, Mode MODE>
__global__ void __launch_bounds__(kThreads) k_bwd(const __grid_constant__ CkptArgs a, uint32_t n, Div row, int nb) {
  grid_dep_wait();
  grid_dep_launch();
  using E = typename Io<DT>::E;
  constexpr int PER = MODE == kOne ? 1 : kPer<DT>;
  const long long blocks = a.M * nb, total = a.M * a.I;
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) {
    const long long at = (long long)i * PER;
    uint32_t c = 0;
    long long b = at / kCkptBlock;
    if (MODE != kFlat) {
      const uint32_t m = quotient(i * PER, row);
      c = i * PER - m * row.d;
      b = (long long)m * nb + c / kCkptBlock;
    }
    const E* dh = static_cast<const E*>(a.dh) + at;
    E *oU = static_cast<E*>(a.dU) + at, *oG = static_cast<E*>(a.dG) + at, *oh = a.h ? static_cast<E*>(a.h) + at : nullptr;
    auto one = [&](int j, float sg, float su) {
      float vU, vG, vh;
      silu_stage<DT>(Io<DT>::ld(dh + j), __fmul_rn((float)a.gq[at + j], sg), __fmul_rn((float)a.uq[at + j], su), vU, vG, vh);
      Io<DT>::st(oU + j, vU);
      Io<DT>::st(oG + j, vG);
      if (oh) Io<DT>::st(oh + j, vh);
    };
    if constexpr (MODE == kOne) {
      one(0, a.gs[b], a.us[b]);
    } else {
      const Scales sg = scales_at<PER, MODE>(a.gs, b, c, a.I, blocks), su = scales_at<PER, MODE>(a.us, b, c, a.I, blocks);
      if (MODE == kMixed && at + PER > total) {   // the array's last elements
        for (int j = 0; at + j < total; ++j) one(j, sg.of(j), su.of(j));
        continue;
      }
      uint32_t qg[PER / 4], qu[PER / 4];
      float d[PER], vU[PER], vG[PER], vh[PER];
      load_vec<DT>(dh, d);
      load_codes<DT>(a.gq + at, qg);
      load_codes<DT>(a.uq + at, qu);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        silu_stage<DT>(d[j], code_value(qg[j / 4], j % 4) * sg.of(j), code_value(qu[j / 4], j % 4) * su.of(j), vU[j], vG[j], vh[j]);
      store_vec<DT>(oU, vU);
      store_vec<DT>(oG, vG);
      if (oh) store_vec<DT>(oh, vh);
    }
  }
}

bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool on8(const void* p) { return ((uintptr_t)p & 7u) == 0; }

// Every launch takes rows enough for less than 2^30 elements (eight rows at
// least, and a multiple of eight, so that vectors stay on their boundaries);
// rows of more elements than 2^27 do not come.
constexpr long long kMost = 1ll << 30;

template <class F>
cudaError_t by_rows(CkptArgs a, F&& launch) {
  const long long nb = (a.I + kCkptBlock - 1) / kCkptBlock, es = a.dtype == DETFFN_F32 ? 4 : 2;
  const long long most = (kMost / a.I) & ~7ll, M = a.M;
  auto skip = [&](auto*& p, long long bytes) {
    if (p) p = reinterpret_cast<std::remove_reference_t<decltype(p)>>((char*)p + bytes);
  };
  for (long long m = 0; m < M; m += most) {
    a.M = M - m < most ? M - m : most;
    const cudaError_t e = launch(a);
    if (e != cudaSuccess) return e;
    const long long n = most * a.I * es;
    skip(a.gate, n);
    skip(a.up, n);
    skip(a.dh, n);
    skip(a.dU, n);
    skip(a.dG, n);
    skip(a.h, n);
    skip(a.gq, most * a.I);
    skip(a.uq, most * a.I);
    skip(a.gs, 4 * most * nb);
    skip(a.us, 4 * most * nb);
  }
  return cudaSuccess;
}

// Up to 64 blocks of threads to an SM, several times what it holds, so that
// SMs that get ahead take more (the backward stage of 4096 x 12288: 86 us with
// as many as it holds, 75.6 so).
int grid_for(long long threads, int sm_count) {
  const long long want = (threads + kThreads - 1) / kThreads, most = (long long)sm_count * 64;
  return (int)(want < most ? want : most);
}

template <int DT>
cudaError_t pack(const CkptArgs& all, int sms, cudaStream_t st) {
  const long long nb = (all.I + kCkptBlock - 1) / kCkptBlock;
  const bool vec = all.I % 8 == 0 && on16(all.gate) && on16(all.up) && on8(all.gq) && on8(all.uq);
  auto k = !vec ? k_pack_any<DT> : all.I % 64 ? k_pack_vec<DT, false> : k_pack_vec<DT, true>;
  return by_rows(all, [&](const CkptArgs& a) {
    return launch_dependent(k, dim3(grid_for(a.M * nb * (vec ? 4 : 8), sms)), kThreads, 0, st, a, (uint32_t)(a.M * nb),
                            div_by((uint32_t)nb));
  });
}

template <int DT>
Mode mode_of(const CkptArgs& a, bool aligned) {
  if (!aligned || a.I < 8) return kOne;
  return a.I % 64 == 0 ? kFlat : a.I % kPer<DT> == 0 ? kRows : kMixed;
}

template <int DT, class F>
cudaError_t by_mode(const CkptArgs& all, Mode mode, int sms, cudaStream_t st, F&& kernel) {
  const int per = mode == kOne ? 1 : kPer<DT>, nb = (int)((all.I + kCkptBlock - 1) / kCkptBlock);
  return by_rows(all, [&](const CkptArgs& a) {
    const long long n = (a.M * a.I + per - 1) / per;
    return launch_dependent(kernel(mode), dim3(grid_for(n, sms)), kThreads, 0, st, a, (uint32_t)n, div_by((uint32_t)a.I), nb);
  });
}

template <int DT>
cudaError_t unpack(const CkptArgs& a, int sms, cudaStream_t st) {
  const Mode mode = mode_of<DT>(a, on16(a.gate) && on16(a.up) && on8(a.gq) && on8(a.uq));
  return by_mode<DT>(a, mode, sms, st, [](Mode m) {
    return m == kFlat ? k_unpack<DT, kFlat> : m == kRows ? k_unpack<DT, kRows> : m == kMixed ? k_unpack<DT, kMixed> : k_unpack<DT, kOne>;
  });
}
template <int DT>
cudaError_t bwd(const CkptArgs& a, int sms, cudaStream_t st) {
  const Mode mode = mode_of<DT>(a, on16(a.dh) && on16(a.dU) && on16(a.dG) && on16(a.h) && on8(a.gq) && on8(a.uq));
  return by_mode<DT>(a, mode, sms, st, [](Mode m) {
    return m == kFlat ? k_bwd<DT, kFlat> : m == kRows ? k_bwd<DT, kRows> : m == kMixed ? k_bwd<DT, kMixed> : k_bwd<DT, kOne>;
  });
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
