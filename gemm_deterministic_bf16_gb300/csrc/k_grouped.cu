// k_grouped.cu -- matrix products grouped by expert on the CUDA cores, for FP32
// and for sizes that the tensor kernel does not take.
//
//   out[r]  = W[e] x[r]            K sums of K products (contraction over the features of x)
//   dx[r]   = W[e]^T dout[r]       (over the features of out)
//   dW[e]   = sum_r dout[r] x[r]^T (over the expert's rows)
//
// All three are D[i, j] = sum_c A(i, c) B(j, c), where A and B run along c or
// across it in memory.  A CTA takes one tile of an expert after another; the
// experts' rows are read on the device, so no host needs to know them.  What bounds
// it is the FP32 multiply-add rate: a thread of a 128 x 128 tile holds 8 x 8 sums and
// reads 16 values of shared memory for each step of c, and the two FP32 multiply-adds
// of fma.rn.f32x2 share an issue slot.  Tiles are 64 x 64 where larger ones would not
// fill the SMs twice; four sets of threads then share the steps of c, for with 4 x 4
// sums a thread is bound by the reads of shared memory (16 experts of 16 rows, K = N =
// 1024, FP32, by such tiles: 124 us, and 75 so).
//
// With few rows of an expert in FP32 the matrices bind, and out and dx have kernels of
// their own that read each once for eight rows.
//
// FP32, 8192 rows of 8 experts, K = 2048, N = 1024: 680 us forward, 602 dx, 627 dW (51 to 57
// TFLOP/s); 777 rows of 5 experts, K = 1031, N = 515: 39, 37 and 36 us.
#include <type_traits>

#include "elt.cuh"
#include "grouped.h"
#include "ptx.cuh"

namespace detffn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Steps of c to a round: more for small tiles, whose arithmetic hides less of the
// loads for the next round.
template <int T> constexpr int kSteps = T == 128 ? 16 : 32;

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}

// An operand tile of T rows (i) and TC columns (c) on its way to shared memory
// s[c][i]; ALONG: memory runs along c.  A thread holds two runs of four
// neighbours in memory, and neighbouring threads a row's.
template <int DT, int T, bool ALONG>
struct Tile {
  using El = typename Io<DT>::E;
  static constexpr int TC = kSteps<T>, RUNS = T * TC / (4 * kThreads);
  static constexpr int PITCH = T + 4;
  static constexpr int LANES = (ALONG ? TC : T) / 4, DOWN = kThreads / LANES;   // threads along memory; rows of a run's threads
  const El* at[RUNS];  // this thread's first elements of the next step
  long long step;
  int i, c, ni;        // its place; rows of the tile that there are
  bool plain;          // all rows, FP32 in whole vectors
  float v[RUNS][4];
  __device__ __forceinline__ int row(int r) const { return ALONG ? i + DOWN * r : i; }
  __device__ __forceinline__ int col(int r) const { return ALONG ? c : c + DOWN * r; }
  // Element (i, c) at p + i * ld + c (ALONG) or p + c * ld + i, for i < ni.
  __device__ __forceinline__ void aim(const El* p, long long ld, long long rows) {
    const int along = (int)threadIdx.x % LANES * 4, down = (int)threadIdx.x / LANES;
    i = ALONG ? down : along;
    c = ALONG ? along : down;
    ni = (int)min(rows, (long long)T);
#pragma unroll
    for (int r = 0; r < RUNS; ++r) at[r] = p + (down + DOWN * r) * ld + along;
    step = ALONG ? TC : TC * ld;
    plain = rows >= T && (DT != DETFFN_F32 || (((uintptr_t)p & 15) == 0 && (ld & 3) == 0));
  }
  // The next TC columns, of which `nc` are there.  PLAIN: all of them, all rows,
  // and FP32 in whole vectors.  (Without branches: each costs a wait for its loads.)
  template <bool PLAIN>
  __device__ __forceinline__ void load(long long nc) {
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if constexpr (PLAIN && DT == DETFFN_F32) {
        *reinterpret_cast<float4*>(v[r]) = *reinterpret_cast<const float4*>(at[r]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[r][u] = 0.0f;
          if (PLAIN || (ALONG ? row(r) < ni && c + u < nc : col(r) < nc && i + u < ni)) v[r][u] = Io<DT>::ld(at[r] + u);
        }
      }
      at[r] += step;
    }
  }
  __device__ __forceinline__ void store(float* s) const {
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      if constexpr (ALONG) {
#pragma unroll
        for (int u = 0; u < 4; ++u) s[(c + u) * PITCH + row(r)] = v[r][u];
      } else {
        *reinterpret_cast<float4*>(s + col(r) * PITCH + i) = *reinterpret_cast<const float4*>(v[r]);
      }
    }
  }
};

// PARTS > 1: the CTAs of a cluster take equal parts of a tile's contraction, and the
// first adds the others' sums in order.
template <int DT, Grouped WHAT, int T, int PARTS>
__global__ void __launch_bounds__(kThreads, 2) k_grouped(const GroupedArgs a) {
  using El = typename Io<DT>::E;
  constexpr bool AA = WHAT != Grouped::kWeight, BA = WHAT == Grouped::kForward;
  constexpr int TC = kSteps<T>;
  constexpr int S = 8, SIDE = T / S, SETS = kThreads / (SIDE * SIDE);   // sums of a thread: S x S
  using TA = Tile<DT, T, AA>;
  using TB = Tile<DT, T, BA>;
  __shared__ __align__(16) float sa[2][TC * TA::PITCH];
  __shared__ __align__(16) float sb[2][TC * TB::PITCH];
  const int set = threadIdx.x / (SIDE * SIDE), ty = threadIdx.x / SIDE % SIDE, tx = threadIdx.x % SIDE;
  const long long J = WHAT == Grouped::kForward ? a.N : a.K;
  const long long tj = (J + T - 1) / T;
  grid_dep_wait();
  grid_dep_launch();
  const int rank = PARTS == 1 ? 0 : (int)cluster_rank();
  long long next = blockIdx.x / PARTS, first = 0;   // this CTA's next tile; the first tile of expert e
  for (int e = 0; e < a.E; ++e) {
    // (Rows out of the tensors, or before the expert's first, are none of its.)
    const long long b = min(max((long long)__ldg(a.off + e), 0ll), a.R);
    const long long n = max(min((long long)__ldg(a.off + e + 1), a.R) - b, 0ll);
    const long long I = WHAT == Grouped::kWeight ? a.N : n;
    const long long all = WHAT == Grouped::kForward ? a.K : WHAT == Grouped::kInput ? a.N : n;
    const long long span = PARTS == 1 ? all : (all + PARTS * TC - 1) / (PARTS * TC) * TC;   // whole rounds
    const long long from = min(rank * span, all), C = min(span, all - from);               // of this CTA
    const long long tiles = (I + T - 1) / T * tj;
    for (; next < first + tiles; next += gridDim.x / PARTS) {
      const long long i0 = (next - first) / tj * T, j0 = (next - first) % tj * T;
      const El* W = static_cast<const El*>(a.W) + (long long)e * a.N * a.K;
      TA ra;
      TB rb;
      if constexpr (WHAT == Grouped::kForward) {
        ra.aim(static_cast<const El*>(a.x.p) + (b + i0) * a.x.ld + from, a.x.ld, I - i0);
        rb.aim(W + j0 * a.K + from, a.K, J - j0);
      } else if constexpr (WHAT == Grouped::kInput) {
        ra.aim(static_cast<const El*>(a.dout.p) + (b + i0) * a.dout.ld + from, a.dout.ld, I - i0);
        rb.aim(W + from * a.K + j0, a.K, J - j0);
      } else {
        ra.aim(static_cast<const El*>(a.dout.p) + (b + from) * a.dout.ld + i0, a.dout.ld, I - i0);
        rb.aim(static_cast<const El*>(a.x.p) + (b + from) * a.x.ld + j0, a.x.ld, J - j0);
      }
      uint64_t sum[S][S / 2];
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < S / 2; ++j) sum[i][j] = 0;
      auto rounds = [&](auto p, long long c0, long long c1) {   // columns c0 .. c1 - 1
        constexpr bool PLAIN = decltype(p)::value;
        ra.template load<PLAIN>(C - c0);
        rb.template load<PLAIN>(C - c0);
        int s = 0;
        for (; c0 < c1; c0 += TC, s ^= 1) {
          ra.store(sa[s]);
          rb.store(sb[s]);
          __syncthreads();   // (the other buffer's readers are past it when it is written again)
          if (c0 + TC < c1) {
            ra.template load<PLAIN>(C - c0 - TC);
            rb.template load<PLAIN>(C - c0 - TC);
          }
#pragma unroll
          for (int k = 0; k < TC / SETS; ++k) {
            // Rows ty * 4 .. + 3 and columns tx * 4 .. + 3 of each half.
            const int c = set * (TC / SETS) + k;
            float x[S];
            uint64_t y[S / 2];
#pragma unroll
            for (int h = 0; h < S / 4; ++h) {
              *reinterpret_cast<float4*>(x + 4 * h) = *reinterpret_cast<const float4*>(sa[s] + c * TA::PITCH + T / 2 * h + 4 * ty);
              *reinterpret_cast<ulonglong2*>(y + 2 * h) = *reinterpret_cast<const ulonglong2*>(sb[s] + c * TB::PITCH + T / 2 * h + 4 * tx);
            }
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
              for (int j = 0; j < S / 2; ++j) sum[i][j] = fma_f32x2(two(x[i], x[i]), y[j], sum[i][j]);
          }
        }
        __syncthreads();   // (the buffers are written again)
      };
      const long long whole = ra.plain && rb.plain ? C / TC * TC : 0;
      if (whole > 0) rounds(std::true_type(), 0, whole);
      if (whole < C) rounds(std::false_type(), whole, C);
      if constexpr (SETS > 1) {   // the sets' sums, in order
        static_assert(sizeof(sa) >= T * T * 4, "one set's sums");
        float* r = &sa[0][0] + threadIdx.x % (SIDE * SIDE);
        for (int other = 1; other < SETS; ++other) {
          if (set == other) {
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
              for (int j = 0; j < S; ++j) r[(i * S + j) * SIDE * SIDE] = __uint_as_float((uint32_t)(sum[i][j / 2] >> (32 * (j % 2))));
          }
          __syncthreads();
          if (set == 0) {
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
              for (int j = 0; j < S / 2; ++j)
                sum[i][j] = add_f32x2(sum[i][j], two(r[(i * S + 2 * j) * SIDE * SIDE], r[(i * S + 2 * j + 1) * SIDE * SIDE]));
          }
          __syncthreads();
        }
        if constexpr (PARTS > 1) {
          for (int other = 1; other < PARTS; ++other) {
            cluster_sync_all();   // (the first CTA is done with its shared memory)
            if (rank == other && set == 0) {
#pragma unroll
              for (int i = 0; i < S; ++i)
#pragma unroll
                for (int j = 0; j < S; ++j)
                  cluster_st(cluster_addr(r + (i * S + j) * SIDE * SIDE, 0), (int)(uint32_t)(sum[i][j / 2] >> (32 * (j % 2))));
            }
            cluster_sync_all();
            if (rank == 0 && set == 0) {
#pragma unroll
              for (int i = 0; i < S; ++i)
#pragma unroll
                for (int j = 0; j < S / 2; ++j)
                  sum[i][j] = add_f32x2(sum[i][j], two(r[(i * S + 2 * j) * SIDE * SIDE], r[(i * S + 2 * j + 1) * SIDE * SIDE]));
            }
          }
          __syncthreads();   // (the buffer is written again)
        }
        if (set > 0 || rank > 0) continue;
      }
      El* out;
      long long lo;
      if constexpr (WHAT == Grouped::kForward) out = static_cast<El*>(const_cast<void*>(a.out.p)) + b * a.out.ld, lo = a.out.ld;
      else if constexpr (WHAT == Grouped::kInput) out = static_cast<El*>(const_cast<void*>(a.dx.p)) + b * a.dx.ld, lo = a.dx.ld;
      else out = static_cast<El*>(a.dW) + (long long)e * a.N * a.K, lo = a.K;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const long long r = i0 + i / 4 * (T / 2) + 4 * ty + i % 4;
        if (r >= I) continue;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const long long c = j0 + j / 4 * (T / 2) + 4 * tx + j % 4;
          if (c < J) Io<DT>::st(out + r * lo + c, __uint_as_float((uint32_t)(sum[i][j / 2] >> (32 * (j % 2)))));
        }
      }
    }
    first += tiles;
  }
}

// out for few rows of an expert, FP32: tiles of four features by eight rows, the
// lanes of a warp along K, so that a matrix is read once for eight rows and nothing
// waits for the rounds of a 64 x 64 tile.  SPLIT warps share a tile's K, 128 in turn:
// all eight of a CTA where there are fewer tiles than warps.  What bounds it is HBM up
// to eight rows (64 experts of one row, K = 2048, N = 768: 79 us, 76 % of the copy rate),
// then the reads of x from L1, twice the matrix's.
// VEC: rows of W and x lie on 16-byte boundaries.
constexpr int kFewRows = 8, kFewFeatures = 4;

template <bool VEC>
__device__ __forceinline__ void few_load(const float* p, int left, int lane, float (&v)[4]) {   // left: of the row from p on
  if constexpr (VEC) {
    const float4 q = 4 * lane < left ? __ldg(reinterpret_cast<const float4*>(p) + lane) : make_float4(0, 0, 0, 0);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = lane + 32 * u < left ? __ldg(p + lane + 32 * u) : 0.0f;
  }
}

// Sums of features f .. f + 3 by ROWS rows at x over this warp's part of K; the lanes
// of feature i and row r, lane / (8 / ROWS) = ROWS * i + r, have its sum.
template <int ROWS, int SPLIT, bool VEC>
__device__ __forceinline__ float few_sums(const float* const (&w)[kFewFeatures], const float* x, long long ldx, int rows, int K,
                                          int part, int lane) {
  constexpr int F = kFewFeatures, STEP = 128 * SPLIT;
  float v[F * ROWS];
#pragma unroll
  for (int i = 0; i < F * ROWS; ++i) v[i] = 0.0f;
  float next[F][4];
  int c = 128 * part;
#pragma unroll
  for (int i = 0; i < F; ++i) few_load<VEC>(w[i] + c, K - c, lane, next[i]);
  for (; c < K; c += STEP) {
    float now[F][4];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) now[i][u] = next[i][u];
    if (c + STEP < K) {
#pragma unroll
      for (int i = 0; i < F; ++i) few_load<VEC>(w[i] + c + STEP, K - c - STEP, lane, next[i]);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      float y[4];
      few_load<VEC>(x + min(r, rows - 1) * ldx + c, K - c, lane, y);   // (a row past the last: its sum is not used)
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) v[ROWS * i + r] = fmaf(now[i][u], y[u], v[ROWS * i + r]);
    }
  }
  // Half of the sums to each half of the lanes, while there are any to halve.
  int n = F * ROWS;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    if (n > 1) {
      n /= 2;
#pragma unroll
      for (int j = 0; j < F * ROWS / 2; ++j)
        if (j < n) {
          const bool up = (lane & d) != 0;
          const float keep = up ? v[j + n] : v[j], send = up ? v[j] : v[j + n];
          v[j] = keep + __shfl_xor_sync(0xffffffffu, send, d);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
    }
  }
  return v[0];
}

// f(expert, group of features, first row, rows) for tiles `next`, next + teams, ... of
// all experts' rows by eights and `groups` groups of features.  All lanes together.
template <class F>
__device__ __forceinline__ void few_tiles(const GroupedArgs& a, long long groups, long long next, long long teams, F&& f) {
  const int lane = threadIdx.x % 32;
  long long first = 0;
  for (int e0 = 0; e0 < a.E; e0 += 32) {   // an expert to a lane
    long long b = 0, n = 0;
    if (e0 + lane < a.E) {   // (rows out of the tensors, or before the expert's first, are none of its)
      b = min(max((long long)__ldg(a.off + e0 + lane), 0ll), a.R);
      n = max(min((long long)__ldg(a.off + e0 + lane + 1), a.R) - b, 0ll);
    }
    const long long tiles = (n + kFewRows - 1) / kFewRows * groups;
    long long end = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end += v;
    }
    end += first;
    first = __shfl_sync(0xffffffffu, end, 31);
    for (; next < first; next += teams) {
      const int owner = __popc(__ballot_sync(0xffffffffu, end <= next));
      const long long tile = next - __shfl_sync(0xffffffffu, end - tiles, owner), chunk = tile / groups;
      const long long r0 = __shfl_sync(0xffffffffu, b, owner) + chunk * kFewRows;
      const int rows = (int)min((long long)kFewRows, __shfl_sync(0xffffffffu, n, owner) - chunk * kFewRows);
      f(e0 + owner, tile - chunk * groups, r0, rows);
    }
  }
}

template <int SPLIT, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) k_grouped_few(const GroupedArgs a) {
  constexpr int F = kFewFeatures;
  static_assert(SPLIT == 1 || SPLIT == kWarps, "a tile to a warp, or to a CTA");
  __shared__ float red[2][kWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = SPLIT == 1 ? 0 : warp, K = (int)a.K;
  grid_dep_wait();
  grid_dep_launch();
  int buf = 0;
  auto tile = [&](int e, long long group, long long r0, int rows) {
    const long long f = group * F;
    const float* w[F];
#pragma unroll
    for (int i = 0; i < F; ++i) w[i] = static_cast<const float*>(a.W) + (e * a.N + min(f + i, a.N - 1)) * a.K;
    const float* x = static_cast<const float*>(a.x.p) + r0 * a.x.ld;
    const bool pair = rows <= 2;
    float v = pair ? few_sums<2, SPLIT, VEC>(w, x, a.x.ld, rows, K, part, lane)
                   : few_sums<kFewRows, SPLIT, VEC>(w, x, a.x.ld, rows, K, part, lane);
    if constexpr (SPLIT > 1) {   // the warps' sums, in order
      red[buf][warp][lane] = v;
      __syncthreads();   // (one a tile: the other buffer's reader is past it when it is written again)
      if (warp == 0) {
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += red[buf][k][lane];
      }
      buf ^= 1;
      if (warp != 0) return;
    }
    const int at = pair ? lane / 4 : lane, i = pair ? at / 2 : at / kFewRows, r = pair ? at % 2 : at % kFewRows;
    if ((!pair || lane % 4 == 0) && r < rows && f + i < a.N)
      static_cast<float*>(const_cast<void*>(a.out.p))[(r0 + r) * a.out.ld + f + i] = v;
  };
  const long long groups = (a.N + F - 1) / F;
  if constexpr (SPLIT == 1) few_tiles(a, groups, (long long)blockIdx.x * kWarps + warp, (long long)gridDim.x * kWarps, tile);
  else few_tiles(a, groups, blockIdx.x, gridDim.x, tile);
}

// dx for few rows of an expert, FP32: a CTA takes tiles of eight rows by 128 columns of
// W, four to a lane (WIDE), or 32, its warps 4 (16) rows of W in turn; dout's values are the
// same for all lanes.  VEC: rows of dout lie on 16-byte boundaries.  Up to two rows
// HBM bounds it (64 experts of one row, K = 2048, N = 768: 82 us, 73 % of the copy rate),
// from there the reads of dout, a vector for 16 multiply-adds of a lane.
template <int ROWS, bool WIDE, bool VEC>
__device__ __forceinline__ void few_inputs(const float* W, long long ldw, int columns, const float* d, long long ldd, int rows,
                                           int N, int warp, int lane, float* red) {
  constexpr int STEP = WIDE ? 4 : 16, U = WIDE ? 4 : 1;   // rows of W at once; columns of a lane
  const bool in = U * lane < columns;
  float next[STEP][U], v[ROWS][U];
  auto load = [&](int n) {
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
      const bool there = in && n + i < N;
      const float* p = W + (n + i) * ldw + U * lane;
      if constexpr (WIDE) {
        const float4 q = there ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0, 0, 0, 0);
        next[i][0] = q.x, next[i][1] = q.y, next[i][2] = q.z, next[i][3] = q.w;
      } else {
        next[i][0] = there ? __ldg(p) : 0.0f;
      }
    }
  };
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int u = 0; u < U; ++u) v[r][u] = 0.0f;
  load(STEP * warp);
  for (int n = STEP * warp; n < N; n += STEP * kWarps) {
    float now[STEP][U];
#pragma unroll
    for (int i = 0; i < STEP; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) now[i][u] = next[i][u];
    if (n + STEP * kWarps < N) load(n + STEP * kWarps);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float* y = d + min(r, rows - 1) * ldd + n;   // (a row past the last: its sums are not used)
#pragma unroll
      for (int i = 0; i < STEP; i += 4) {
        float q[4] = {};
        if constexpr (VEC) {
          if (n + i < N) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(y + i));
            q[0] = f.x, q[1] = f.y, q[2] = f.z, q[3] = f.w;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (n + i + k < N) q[k] = __ldg(y + i + k);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int u = 0; u < U; ++u) v[r][u] = fmaf(q[k], now[i + k][u], v[r][u]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int u = 0; u < U; ++u) red[r * 32 * U + 32 * u + lane] = v[r][u];
}

template <bool WIDE, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) k_grouped_few_inputs(const GroupedArgs a) {
  constexpr int U = WIDE ? 4 : 1, COLUMNS = 32 * U;
  __shared__ float red[kWarps][kFewRows * COLUMNS];   // [row][column of the lanes][lane]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, N = (int)a.N;
  grid_dep_wait();
  grid_dep_launch();
  few_tiles(a, (a.K + COLUMNS - 1) / COLUMNS, blockIdx.x, gridDim.x, [&](int e, long long group, long long r0, int rows) {
    const long long k0 = group * COLUMNS;
    const int columns = (int)min((long long)COLUMNS, a.K - k0);
    const float *W = static_cast<const float*>(a.W) + e * a.N * a.K + k0,
                *d = static_cast<const float*>(a.dout.p) + r0 * a.dout.ld;
    __syncthreads();   // (the readers of the last tile's sums)
    if (rows <= 2) few_inputs<2, WIDE, VEC>(W, a.K, columns, d, a.dout.ld, rows, N, warp, lane, red[warp]);
    else few_inputs<kFewRows, WIDE, VEC>(W, a.K, columns, d, a.dout.ld, rows, N, warp, lane, red[warp]);
    __syncthreads();
    for (int o = threadIdx.x; o < rows * COLUMNS; o += kThreads) {   // the warps' sums, in order
      const int r = o / COLUMNS, c = o % COLUMNS;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[w][r * COLUMNS + c % U * 32 + c / U];
      if (c < columns) static_cast<float*>(const_cast<void*>(a.dx.p))[(r0 + r) * a.dx.ld + k0 + c] = v;
    }
  });
}

// Tiles of eight rows that there are at least, where experts have rows alike.
long long few_chunks(const GroupedArgs& a) {
  const long long reached = a.R < a.E ? a.R : a.E, chunks = a.R / kFewRows;
  return reached > chunks ? reached : chunks;
}

cudaError_t run_few_inputs(const GroupedArgs& a, int sm_count, cudaStream_t st) {
  // Narrow tiles where wide ones leave SMs without any.
  const bool wide = a.K % 4 == 0 && (uintptr_t)a.W % 16 == 0 && few_chunks(a) * ((a.K + 127) / 128) >= sm_count;
  const bool vec = a.N % 4 == 0 && (uintptr_t)a.dout.p % 16 == 0 && (a.R <= 1 || a.dout.ld % 4 == 0);
  const dim3 grid(2 * sm_count);
  auto go = [&](auto* kernel) { return launch_dependent(kernel, grid, kThreads, 0, st, a); };
  if (wide) return vec ? go(k_grouped_few_inputs<true, true>) : go(k_grouped_few_inputs<true, false>);
  return vec ? go(k_grouped_few_inputs<false, true>) : go(k_grouped_few_inputs<false, false>);
}

cudaError_t run_few(const GroupedArgs& a, int sm_count, cudaStream_t st) {
  const bool vec = a.K % 4 == 0 && (uintptr_t)a.W % 16 == 0 && (uintptr_t)a.x.p % 16 == 0 && (a.R <= 1 || a.x.ld % 4 == 0);
  const long long groups = (a.N + kFewFeatures - 1) / kFewFeatures, tiles = few_chunks(a) * groups,
                  warps = 2ll * sm_count * kWarps;
  const dim3 grid(2 * sm_count);
  auto go = [&](auto* kernel) { return launch_dependent(kernel, grid, kThreads, 0, st, a); };
  if (tiles < warps) return vec ? go(k_grouped_few<kWarps, true>) : go(k_grouped_few<kWarps, false>);
  return vec ? go(k_grouped_few<1, true>) : go(k_grouped_few<1, false>);
}

template <int DT, Grouped WHAT>
cudaError_t run(const GroupedArgs& a, int sm_count, cudaStream_t st) {
  const long long J = WHAT == Grouped::kForward ? a.N : a.K;
  // Tiles of T x T, taking an expert's rows as the average.
  auto tiles = [&](long long T) {
    const long long rows = (a.R + a.E - 1) / a.E;
    return a.E * (((WHAT == Grouped::kWeight ? a.N : rows) + T - 1) / T) * ((J + T - 1) / T);
  };
  auto most = [&](long long T) {
    return (WHAT == Grouped::kWeight ? a.E * ((a.N + T - 1) / T) : a.R / T + a.E) * ((J + T - 1) / T);
  };
  const bool small = tiles(128) < 2ll * sm_count || (WHAT != Grouped::kWeight && a.R <= 64ll * a.E);
  const long long n = most(small ? 64 : 128), slots = 2ll * sm_count;
  // FP32, and no more small tiles than half (a quarter) of the CTAs that there is room for:
  // clusters of two (four) take a tile each, where a contraction has rounds enough to
  // share: 777 rows of 5 experts, K = 1031, N = 515 44 and 39 us; 300 rows, K = N = 512 23 and
  // 15 (with four 16); 256 rows of 4 experts, K = N = 1024 34, 33 and 22; dW of 2000 rows, K
  // = N = 128 60, 35 and 22.
  if constexpr (DT == DETFFN_F32) {
    const long long c = WHAT == Grouped::kForward ? a.K : WHAT == Grouped::kInput ? a.N : a.R / a.E;
    auto parts = [&](auto* kernel, long long p) {
      const long long clusters = n < slots / p ? n : slots / p;
      return launch_cluster(kernel, dim3((unsigned)(p * clusters)), kThreads, 0, (int)p, st, a);
    };
    if (small && 4 * tiles(64) <= slots && c >= 1024) return parts(k_grouped<DT, WHAT, 64, 4>, 4);
    if (small && 2 * tiles(64) <= slots && c > 64) return parts(k_grouped<DT, WHAT, 64, 2>, 2);
  }
  const dim3 grid((unsigned)(n < slots ? n : slots));
  return small ? launch_dependent(k_grouped<DT, WHAT, 64, 1>, grid, kThreads, 0, st, a)
               : launch_dependent(k_grouped<DT, WHAT, 128, 1>, grid, kThreads, 0, st, a);
}

template <int DT>
cudaError_t run(const GroupedArgs& a, Grouped what, int sm_count, cudaStream_t st) {
  if (what == Grouped::kForward) return run<DT, Grouped::kForward>(a, sm_count, st);
  if (what == Grouped::kInput) return run<DT, Grouped::kInput>(a, sm_count, st);
  return run<DT, Grouped::kWeight>(a, sm_count, st);
}

// The y-th expert that has rows, or -1.  All lanes together.
__device__ __forceinline__ int reached(const int* off, int E, long long R, int y) {
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + (int)threadIdx.x % 32;
    uint32_t has = __ballot_sync(0xffffffffu, e < E && min((long long)__ldg(off + e + 1), R) > max((long long)__ldg(off + e), 0ll));
    if (y < __popc(has)) {
      for (; y > 0; --y) has &= has - 1;
      return e0 + __ffs(has) - 1;
    }
    y -= __popc(has);
  }
  return -1;
}

// Eight elements of a row to a thread: aligned words (of a row that begins in the
// middle of one, shifted by half), whose loads cost a quarter of the elements'.
// REACHED: of E matrices, CTAs (.., y) take that of the y-th expert that has rows.
template <bool REACHED>
__global__ void __launch_bounds__(256) k_rows(const uint16_t* all, long long ld, long long rows, long long width, uint16_t* to_all,
                                              const int* off, int E, long long R) {
  const long long per = (width + 7) / 8, n = rows * per;
  grid_dep_wait();
  grid_dep_launch();
  for (int y = blockIdx.y;; y += gridDim.y) {   // (more than there are rows only where ends are out of order)
    const int m = REACHED ? reached(off, E, R, y) : 0;
    if (m < 0) return;
    const uint16_t* from = REACHED ? all + m * rows * ld : all;
    uint16_t* to = REACHED ? to_all + m * n * 8 : to_all;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += 256ll * gridDim.x) {
      const long long r = i / per, c = (i - r * per) * 8;
      const uint16_t* p = from + r * ld + c;
      uint32_t w[4];
      if (c + 8 <= width) {
        const bool odd = ((uintptr_t)p & 2) != 0;
        const uint32_t* q = reinterpret_cast<const uint32_t*>((uintptr_t)p & ~(uintptr_t)3);
        uint32_t v[5];
        v[0] = odd ? (uint32_t)p[0] << 16 : __ldg(q);   // (the word may begin before the tensor)
#pragma unroll
        for (int k = 1; k < 4; ++k) v[k] = __ldg(q + k);
        v[4] = odd ? p[7] : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = odd ? __funnelshift_r(v[k], v[k + 1], 16) : v[k];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = (c + 2 * k < width ? p[2 * k] : 0u) | (c + 2 * k + 1 < width ? (uint32_t)p[2 * k + 1] << 16 : 0u);
      }
      reinterpret_cast<uint4*>(to)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (!REACHED) return;
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_grouped_rows(const Rows& from, long long rows, long long width, uint16_t* to, int sm_count, cudaStream_t st) {
  const long long n = (rows * ((width + 7) / 8) + 255) / 256, most = 16ll * sm_count;
  return launch_dependent(k_rows<false>, dim3((unsigned)(n < most ? n : most)), 256, 0, st, static_cast<const uint16_t*>(from.p),
                          from.ld, rows, width, to, nullptr, 1, 0);
}

cudaError_t launch_grouped_matrices(const GroupedArgs& a, uint16_t* to, int sm_count, cudaStream_t st) {
  // Fewer rows than experts leave some without any, whose matrices nothing reads.  (BF16, K =
  // 2047, N = 1023, out: one row and 256 experts 451 us with all of them laid out and 26 so, 8
  // rows and 64 experts 123 and 33.)
  if (a.R >= a.E) return launch_grouped_rows(Rows{a.W, a.ldw}, a.E * a.N, a.K, to, sm_count, st);
  const long long n = (a.N * ((a.K + 7) / 8) + 255) / 256, most = (16ll * sm_count + a.R - 1) / a.R;
  return launch_dependent(k_rows<true>, dim3((unsigned)(n < most ? n : most), (unsigned)a.R), 256, 0, st,
                          static_cast<const uint16_t*>(a.W), a.ldw, a.N, a.K, to, a.off, a.E, a.R);
}

cudaError_t launch_grouped_general(const GroupedArgs& a, Grouped what, int sm_count, cudaStream_t st) {
  // Tiles of 64 x 64 take what K's rounds of loads do however few rows there are, rows by
  // eights as long as there are eights.  64 experts of 8, 16, 24, 32 and 40 rows, K = 2048, N = 768:
  // 418 us by tiles, 119, 212, 314, 408 and 508 by eights; 16 of 24, 32 and 48, K = N = 1024: 77, and 56,
  // 72 and 110; one of 64, 256 and 384, K = 1024, N = 512: 14, 21 and 22, and 9, 16 and 23.  (The rows are
  // taken as the experts' alike.  1024 that are all one's of 64, K = 2048, N = 768: 124 and 133.)
  if (a.dtype == DETFFN_F32 && what == Grouped::kForward && (a.R <= 32ll * a.E || a.R * a.N <= 1 << 17))
    return run_few(a, sm_count, st);
  // dx of the same: 345, and 134, 243, 353, 456 and 582; 68, and 65, 74 and 131; 12, 17 and 18, and 9, 15
  // and 28; 91 and 134.
  if (a.dtype == DETFFN_F32 && what == Grouped::kInput && (a.R <= 24ll * a.E || a.R * a.K <= 1 << 16))
    return run_few_inputs(a, sm_count, st);
  if (a.dtype == DETFFN_F32) return run<DETFFN_F32>(a, what, sm_count, st);
  if (a.dtype == DETFFN_F16) return run<DETFFN_F16>(a, what, sm_count, st);
  return run<DETFFN_BF16>(a, what, sm_count, st);
}

}  // namespace detffn
