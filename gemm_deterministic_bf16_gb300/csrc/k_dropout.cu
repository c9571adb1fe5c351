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
//
// HBM bounds it with a residual or in FP32 (16384 x 4096: BF16 70 us with a residual, 86 %
// of the copy rate; FP32 89 us without, 90 %).  Where bytes are fewer it is the latency
// of the ten rounds, each of which waits for the last: 20 wide multiplications and 20
// logic operations for four elements keep their pipes at 40 and 64 %, issue is at 55 and
// HBM at 43, and none is full (BF16 without a residual 62 us, 65 %; rows of 4095 94 us,
// element by element).
#include "dropout.h"
#include "elt.cuh"

namespace detffn {
namespace {

// The keys of the ten rounds.  Formed anew for each counter they are a third of
// its instructions: they are kernel arguments, or, with a seed on the device,
// kept in registers.
struct Keys {
  uint32_t a[10], b[10];
};
__host__ __device__ inline Keys keys_of(unsigned long long seed) {
  Keys k;
  for (int r = 0; r < 10; ++r) {
    k.a[r] = (uint32_t)seed + (uint32_t)r * 0x9E3779B9u;
    k.b[r] = (uint32_t)(seed >> 32) + (uint32_t)r * 0xBB67AE85u;
  }
  return k;
}
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, const Keys& k) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k.a[r];
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k.b[r];
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Eight elements as they are stored.
template <int DT> struct Raw {
  static constexpr int N = Io<DT>::kBytes / 2;
  uint4 q[N];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = static_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const { Io<DT>::ld8(reinterpret_cast<const typename Io<DT>::E*>(q), v); }
};

// A thread takes a unit of W features of a row (8 where rows are whole 16-byte
// vectors, loaded while the unit before is worked on; else 4), then the one a
// grid further on.
template <int DT, int W, bool RES, bool STATE>
__global__ void __launch_bounds__(256) k_dropout(const DropoutArgs a, const Keys given) {
  using El = typename Io<DT>::E;
  const long long per = (a.H + W - 1) / W, step = (long long)gridDim.x * 256, u = (long long)blockIdx.x * 256 + threadIdx.x;
  long long m = u / per, c = u - m * per;
  const long long dm = step / per, dc = step - dm * per;
  grid_dep_wait();
  grid_dep_launch();
  unsigned long long offset = a.offset;
  Keys own;
  if constexpr (STATE) {
    own = keys_of(a.state[0]);
    offset += a.state[1];
#pragma unroll
    for (int r = 0; r < 10; ++r) asm volatile("" : "+r"(own.a[r]), "+r"(own.b[r]));   // (or they are formed anew)
  }
  const Keys& keys = STATE ? own : given;
  const uint32_t o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
  const El* x = static_cast<const El*>(a.x.p);
  const El* res = static_cast<const El*>(a.residual.p);
  El* out = static_cast<El*>(const_cast<void*>(a.out.p));
  constexpr bool AHEAD = W == 8 && DT == DETFFN_F32;
  Raw<DT> nx, nr;
  auto ahead = [&]() {
    if constexpr (AHEAD) {
      if (m < a.M) {
        nx.load(x + m * a.x.ld + 8 * c);
        if constexpr (RES) nr.load(res + m * a.residual.ld + 8 * c);
      }
    }
  };
  ahead();
  while (m < a.M) {
    const long long f = c * W;
    const uint32_t row = (uint32_t)m;
    El* to = out + m * a.out.ld + f;
    float v[W], r[W];
    if constexpr (AHEAD) {
      nx.values(v);
      if constexpr (RES) nr.values(r);
    } else if constexpr (W == 8) {
      Io<DT>::ld8(x + m * a.x.ld + f, v);
      if constexpr (RES) Io<DT>::ld8(res + m * a.residual.ld + f, r);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[i] = f + i < a.H ? Io<DT>::ld(x + m * a.x.ld + f + i) : 0.0f;
        if constexpr (RES) r[i] = f + i < a.H ? Io<DT>::ld(res + m * a.residual.ld + f + i) : 0.0f;
      }
    }
    m += dm;
    c += dc;
    if (c >= per) {
      c -= per;
      ++m;
    }
    ahead();
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 q = philox((uint32_t)((f + i) >> 2), row, o0, o1, keys);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i + j] = w[j] >= a.limit ? v[i + j] * a.scale : 0.0f;
        if constexpr (RES) v[i + j] = __fadd_rn(r[i + j], v[i + j]);
      }
    }
    if constexpr (W == 8) {
      Io<DT>::st8(to, v);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (f + i < a.H) Io<DT>::st(to + i, v[i]);
    }
  }
}

template <int DT, int W>
cudaError_t run(const DropoutArgs& a, dim3 grid, cudaStream_t st) {
  if (a.none) {   // nothing is kept
    const size_t es = Io<DT>::kBytes, row = (size_t)a.H * es, to = a.M > 1 ? (size_t)a.out.ld * es : row;
    void* out = const_cast<void*>(a.out.p);
    if (!a.residual.p) return cudaMemset2DAsync(out, to, 0, row, (size_t)a.M, st);
    if (a.residual.p == out) return cudaSuccess;
    return cudaMemcpy2DAsync(out, to, a.residual.p, a.M > 1 ? (size_t)a.residual.ld * es : row, row, (size_t)a.M,
                             cudaMemcpyDeviceToDevice, st);
  }
  const Keys k = keys_of(a.seed);
  if (a.state)
    return a.residual.p ? launch_dependent(k_dropout<DT, W, true, true>, grid, 256, 0, st, a, k)
                        : launch_dependent(k_dropout<DT, W, false, true>, grid, 256, 0, st, a, k);
  return a.residual.p ? launch_dependent(k_dropout<DT, W, true, false>, grid, 256, 0, st, a, k)
                      : launch_dependent(k_dropout<DT, W, false, false>, grid, 256, 0, st, a, k);
}

template <int DT>
cudaError_t run(const DropoutArgs& a, int sm_count, cudaStream_t st) {
  const Rows* rows[] = {&a.x, &a.residual, &a.out};
  const long long es = Io<DT>::kBytes;
  bool vec = a.H % 8 == 0;
  for (const Rows* r : rows)
    if (r->p && ((uintptr_t)r->p % 16 != 0 || (a.M > 1 && r->ld * es % 16 != 0))) vec = false;
  const long long W = vec ? 8 : 4, units = a.M * ((a.H + W - 1) / W), most = 8ll * sm_count, want = (units + 255) / 256;
  const dim3 grid((unsigned)(want < most ? want : most));
  return vec ? run<DT, 8>(a, grid, st) : run<DT, 4>(a, grid, st);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int sm_count, cudaStream_t st) {
  if (a.dtype == DETFFN_F32) return run<DETFFN_F32>(a, sm_count, st);
  if (a.dtype == DETFFN_F16) return run<DETFFN_F16>(a, sm_count, st);
  return run<DETFFN_BF16>(a, sm_count, st);
}

}  // namespace detffn
