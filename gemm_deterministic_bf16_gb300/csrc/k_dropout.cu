// k_dropout.cu -- dropout whose mask is formed from a counter and never stored.
//
//   word(m, c) = word c mod 4 of Philox4x32-10 of the counter (c / 4, m,
//                offset low, offset high) under the key (seed low, seed high)
//   out        = residual + (word(m, c) >= floor(p 2^32) ? x / (1 - p) : 0)
//
// Philox4x32-10: J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011.  Each row starts a counter of
// its own, so an element's word depends on its place alone, whatever the width,
// the strides or the other rows are, and the backward pass forms the same mask
// again from two numbers.
//
// A word is 32 bits, so p is met to 2^-32.  The product x * scale and the sum
// are FP32, rounded once to the stored type.
#include "dropout.h"
#include "elt.cuh"

namespace detffn {
namespace {

__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// A thread takes a unit of W features of a row (8 where rows are whole 16-byte
// vectors, else 4) and then the unit a grid further on.
template <int DT, int W, bool RES>
__global__ void __launch_bounds__(256) k_dropout(const DropoutArgs a) {
  using El = typename Io<DT>::E;
  const long long per = (a.H + W - 1) / W, step = (long long)gridDim.x * 256, u = (long long)blockIdx.x * 256 + threadIdx.x;
  long long m = u / per, c = u - m * per;
  const long long dm = step / per, dc = step - dm * per;
  grid_dep_wait();
  grid_dep_launch();
  unsigned long long seed = a.seed, offset = a.offset;
  if (a.state) {
    seed = a.state[0];
    offset += a.state[1];
  }
  const uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32), o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
  const El* x = static_cast<const El*>(a.x.p);
  const El* res = static_cast<const El*>(a.residual.p);
  El* out = static_cast<El*>(const_cast<void*>(a.out.p));
  while (m < a.M) {
    const long long f = c * W;
    float v[W];
    if constexpr (W == 8) {
      Io<DT>::ld8(x + m * a.x.ld + f, v);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = f + i < a.H ? Io<DT>::ld(x + m * a.x.ld + f + i) : 0.0f;
    }
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 q = philox((uint32_t)((f + i) >> 2), (uint32_t)m, o0, o1, k0, k1);
      w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = w[i] >= a.limit && !a.none ? v[i] * a.scale : 0.0f;
    if constexpr (RES) {
      float r[W];
      if constexpr (W == 8) {
        Io<DT>::ld8(res + m * a.residual.ld + f, r);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) r[i] = f + i < a.H ? Io<DT>::ld(res + m * a.residual.ld + f + i) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = __fadd_rn(r[i], v[i]);
    }
    if constexpr (W == 8) {
      Io<DT>::st8(out + m * a.out.ld + f, v);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (f + i < a.H) Io<DT>::st(out + m * a.out.ld + f + i, v[i]);
    }
    m += dm;
    c += dc;
    if (c >= per) {
      c -= per;
      ++m;
    }
  }
}

template <int DT>
cudaError_t run(const DropoutArgs& a, int sm_count, cudaStream_t st) {
  const Rows* rows[] = {&a.x, &a.residual, &a.out};
  const long long es = Io<DT>::kBytes;
  bool vec = a.H % 8 == 0;
  for (const Rows* r : rows)
    if (r->p && ((uintptr_t)r->p % 16 != 0 || (a.M > 1 && r->ld * es % 16 != 0))) vec = false;
  const int W = vec ? 8 : 4;
  const long long units = a.M * ((a.H + W - 1) / W), most = 8ll * sm_count;
  const long long want = (units + 255) / 256;
  const dim3 grid((unsigned)(want < most ? want : most));
  if (vec)
    return a.residual.p ? launch_dependent(k_dropout<DT, 8, true>, grid, 256, 0, st, a)
                        : launch_dependent(k_dropout<DT, 8, false>, grid, 256, 0, st, a);
  return a.residual.p ? launch_dependent(k_dropout<DT, 4, true>, grid, 256, 0, st, a)
                      : launch_dependent(k_dropout<DT, 4, false>, grid, 256, 0, st, a);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int sm_count, cudaStream_t st) {
  if (a.dtype == DETFFN_F32) return run<DETFFN_F32>(a, sm_count, st);
  if (a.dtype == DETFFN_F16) return run<DETFFN_F16>(a, sm_count, st);
  return run<DETFFN_BF16>(a, sm_count, st);
}

}  // namespace detffn
