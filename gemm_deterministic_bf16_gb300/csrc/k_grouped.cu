// k_grouped.cu -- matrix products grouped by expert on the CUDA cores, for FP32
// and for sizes that the tensor kernel does not take.
//
//   out[r]  = W[e] x[r]            K sums of K products (contraction over the features of x)
//   dx[r]   = W[e]^T dout[r]       (over the features of out)
//   dW[e]   = sum_r dout[r] x[r]^T (over the expert's rows)
//
// All three are D[i, j] = sum_c A(i, c) B(j, c), where A and B run along c or
// across it in memory.  A CTA takes a tile of TI x 128 of one expert after
// another; the experts' rows are read on the device, so no host needs to know
// them.  What bounds it is the FP32 multiply-add rate: a thread holds TI / 16 x
// 8 sums and reads TI / 16 + 8 values of shared memory for each step of c, and
// the two FP32 multiply-adds of fma.rn.f32x2 share an issue slot.
#include "elt.cuh"
#include "grouped.h"

namespace detffn {
namespace {

constexpr int TJ = 128, TC = 16, kThreads = 256;

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}

// An operand tile of T rows (i) and TC columns (c) on its way to shared memory
// s[c][i]: ALONG, memory runs along c.  A thread holds T * TC / 256 values.
template <int DT, int T, bool ALONG>
struct Tile {
  using El = typename Io<DT>::E;
  static constexpr int V = T * TC / kThreads;   // 8 (T = 128) or 2 (T = 32)
  static constexpr int PITCH = T + 4;
  float v[V];
  __device__ __forceinline__ static int i_of(int u) {
    return ALONG ? (u * kThreads + (int)threadIdx.x) / TC : (u * kThreads + (int)threadIdx.x) % T;
  }
  __device__ __forceinline__ static int c_of(int u) {
    return ALONG ? (u * kThreads + (int)threadIdx.x) % TC : (u * kThreads + (int)threadIdx.x) / T;
  }
  // Element (i, c) at p + i * ld + c (ALONG) or p + c * ld + i; zero from ni, nc on.
  __device__ __forceinline__ void load(const El* p, long long ld, long long ni, long long nc) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int i = i_of(u), c = c_of(u);
      v[u] = i < ni && c < nc ? Io<DT>::ld(p + (ALONG ? i * ld + c : c * ld + i)) : 0.0f;
    }
  }
  __device__ __forceinline__ void store(float* s) const {
#pragma unroll
    for (int u = 0; u < V; ++u) s[c_of(u) * PITCH + i_of(u)] = v[u];
  }
};

template <int DT, Grouped WHAT, int TI>
__global__ void __launch_bounds__(kThreads) k_grouped(const GroupedArgs a) {
  using El = typename Io<DT>::E;
  constexpr bool AA = WHAT != Grouped::kWeight, BA = WHAT == Grouped::kForward;
  constexpr int RI = TI / 16;                    // sums of a thread: RI x 8
  using TA = Tile<DT, TI, AA>;
  using TB = Tile<DT, TJ, BA>;
  __shared__ __align__(16) float sa[2][TC * TA::PITCH];
  __shared__ __align__(16) float sb[2][TC * TB::PITCH];
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const long long J = WHAT == Grouped::kForward ? a.N : a.K;
  const long long tj = (J + TJ - 1) / TJ;
  grid_dep_wait();
  grid_dep_launch();
  long long next = blockIdx.x, first = 0;        // this CTA's next tile; the first tile of expert e
  for (int e = 0; e < a.E; ++e) {
    // (Rows out of the tensors, or before the expert's first, are none of its.)
    const long long b = min(max((long long)__ldg(a.off + e), 0ll), a.R);
    const long long n = max(min((long long)__ldg(a.off + e + 1), a.R) - b, 0ll);
    const long long I = WHAT == Grouped::kWeight ? a.N : n;
    const long long C = WHAT == Grouped::kForward ? a.K : WHAT == Grouped::kInput ? a.N : n;
    const long long tiles = (I + TI - 1) / TI * tj;
    for (; next < first + tiles; next += gridDim.x) {
      const long long i0 = (next - first) / tj * TI, j0 = (next - first) % tj * TJ;
      const El* W = static_cast<const El*>(a.W) + (long long)e * a.N * a.K;
      // A(i, c) and B(j, c) of this tile.
      const El *pa, *pb;
      long long la, lb;
      if constexpr (WHAT == Grouped::kForward) {
        pa = static_cast<const El*>(a.x.p) + (b + i0) * a.x.ld, la = a.x.ld;
        pb = W + j0 * a.K, lb = a.K;
      } else if constexpr (WHAT == Grouped::kInput) {
        pa = static_cast<const El*>(a.dout.p) + (b + i0) * a.dout.ld, la = a.dout.ld;
        pb = W + j0, lb = a.K;
      } else {
        pa = static_cast<const El*>(a.dout.p) + b * a.dout.ld + i0, la = a.dout.ld;
        pb = static_cast<const El*>(a.x.p) + b * a.x.ld + j0, lb = a.x.ld;
      }
      uint64_t sum[RI][4];
#pragma unroll
      for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = 0;
      TA ra;
      TB rb;
      ra.load(pa, la, I - i0, C);
      rb.load(pb, lb, J - j0, C);
      int s = 0;
      for (long long c0 = 0; c0 < C; c0 += TC, s ^= 1) {
        ra.store(sa[s]);
        rb.store(sb[s]);
        __syncthreads();   // (the other buffer's readers are past it when it is written again)
        if (c0 + TC < C) {
          ra.load(pa + (AA ? c0 + TC : (c0 + TC) * la), la, I - i0, C - c0 - TC);
          rb.load(pb + (BA ? c0 + TC : (c0 + TC) * lb), lb, J - j0, C - c0 - TC);
        }
#pragma unroll
        for (int c = 0; c < TC; ++c) {
          float x[RI];
          uint64_t y[4];
          const float* fa = sa[s] + c * TA::PITCH;
          const float* fb = sb[s] + c * TB::PITCH;
          // Rows ty * 4 .. + 3 of each 64 (or two of 32); columns tx * 4 .. + 3 of each 64.
          if constexpr (RI == 8) {
            *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(fa + 4 * ty);
            *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(fa + 64 + 4 * ty);
          } else {
#pragma unroll
            for (int i = 0; i < RI; ++i) x[i] = fa[RI * ty + i];
          }
          *reinterpret_cast<ulonglong2*>(y) = *reinterpret_cast<const ulonglong2*>(fb + 4 * tx);
          *reinterpret_cast<ulonglong2*>(y + 2) = *reinterpret_cast<const ulonglong2*>(fb + 64 + 4 * tx);
#pragma unroll
          for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[i][j] = fma_f32x2(two(x[i], x[i]), y[j], sum[i][j]);
        }
      }
      __syncthreads();   // (the next tile writes the buffers)
      El* out;
      long long lo;
      if constexpr (WHAT == Grouped::kForward) out = static_cast<El*>(const_cast<void*>(a.out.p)) + b * a.out.ld, lo = a.out.ld;
      else if constexpr (WHAT == Grouped::kInput) out = static_cast<El*>(const_cast<void*>(a.dx.p)) + b * a.dx.ld, lo = a.dx.ld;
      else out = static_cast<El*>(a.dW) + (long long)e * a.N * a.K, lo = a.K;
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const long long r = i0 + (RI == 8 ? i / 4 * 64 + 4 * ty + i % 4 : RI * ty + i);
        if (r >= I) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const long long c = j0 + j / 4 * 64 + 4 * tx + j % 4;
          if (c < J) Io<DT>::st(out + r * lo + c, __uint_as_float((uint32_t)(sum[i][j / 2] >> (32 * (j % 2)))));
        }
      }
    }
    first += tiles;
  }
}

template <int DT, Grouped WHAT>
cudaError_t run(const GroupedArgs& a, int sm_count, cudaStream_t st) {
  // Rows of the tile: 32 where an expert has that many on average, or fewer;
  // 128 would then multiply padding.
  const long long I = WHAT == Grouped::kWeight ? a.N : (a.R + a.E - 1) / a.E;
  const long long J = WHAT == Grouped::kForward ? a.N : a.K;
  const bool few = I <= 32;
  const int TI = few ? 32 : 128;
  const long long most = (WHAT == Grouped::kWeight ? a.E * ((a.N + TI - 1) / TI) : a.R / TI + a.E) * ((J + TJ - 1) / TJ);
  const long long slots = 2ll * sm_count;
  const dim3 grid((unsigned)(most < slots ? most : slots));
  return few ? launch_dependent(k_grouped<DT, WHAT, 32>, grid, kThreads, 0, st, a)
             : launch_dependent(k_grouped<DT, WHAT, 128>, grid, kThreads, 0, st, a);
}

template <int DT>
cudaError_t run(const GroupedArgs& a, Grouped what, int sm_count, cudaStream_t st) {
  if (what == Grouped::kForward) return run<DT, Grouped::kForward>(a, sm_count, st);
  if (what == Grouped::kInput) return run<DT, Grouped::kInput>(a, sm_count, st);
  return run<DT, Grouped::kWeight>(a, sm_count, st);
}

}  // namespace

cudaError_t launch_grouped_general(const GroupedArgs& a, Grouped what, int sm_count, cudaStream_t st) {
  if (a.dtype == DETFFN_F32) return run<DETFFN_F32>(a, what, sm_count, st);
  if (a.dtype == DETFFN_F16) return run<DETFFN_F16>(a, what, sm_count, st);
  return run<DETFFN_BF16>(a, what, sm_count, st);
}

}  // namespace detffn
