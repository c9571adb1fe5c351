// k_w4.cu -- products of a few tokens with matrices of 4-bit codes and a scale
// for each group of 32, 64 or 128 codes of a row.
//
//   y[t, n] = sum over groups g of  s[n, g] * ( sum over k in g of (code[n, k] - 8) * x[t, k] )
//
// What bounds it is the weights' bytes (half a byte a weight and the scales).
// At the card's copy rate an SM has to take in some 46 weights a cycle, so
// the arithmetic goes to the tensor cores by mma.sync m16n8k16, straight from
// registers: the weights are the 16-row operand, up to eight columns (tokens,
// or the terms of their activations) the other, and a weight is read and
// converted once for all of them.  A code becomes BF16 or FP16 by putting its
// bits into the mantissa of 128 or 1024 and subtracting 136 or 1032: exact, as
// are all products with a 16-bit x.  A group's sum is one accumulation in FP32,
// scaled and added to the row's FP32 sum.
//
// An FP32 activation is three BF16 terms (each the leading eight bits of what
// the ones before left, together all 24), in columns of their own.  The hidden
// activation of the gated FFN goes from one launch to the next in FP32, and as
// two terms (16 bits) where the result is a 16-bit type.
//
// The order of the codes makes this a matter of plain vectors: lane 4 r + t of
// a warp holds row r (and r + 8) of the 16-row operand and columns 2 t, 2 t + 1,
// 2 t + 8, 2 t + 9 of each 16 of K.  As any order of K serves, chunk t of a run
// of 128 codes (16 bytes) holds what lane t needs of it: word g the codes 32 g +
// 8 t .. + 7 of group quarter g, nibble p of it code 2 (p mod 4) + p / 4, so
// that a mask and a shift leave neighbours in the two halves of a register.
#include "elt.cuh"
#include "w4.h"

namespace detffn {
namespace {

constexpr int kWarps = 8;

template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes 2 i and 2 i + 1 of a word, less 8, in the halves of a register.
template <bool BF16>
__device__ __forceinline__ uint32_t pair(uint32_t word, int i) {
  const uint32_t v = word >> (4 * i) & 0x000F000Fu;
  uint32_t r;
  if constexpr (BF16) {
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v | 0x43004300u), "r"(0x43084308u));  // 128 + code - 136
  } else {
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v | 0x64006400u), "r"(0x64086408u));   // 1024 + code - 1032
  }
  return r;
}

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float ld_scale(const void* p, long long i, int type) {
  if (type == DETFFN_F32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t v = __ldg(static_cast<const uint16_t*>(p) + i);
  return type == DETFFN_F16 ? __half2float(__ushort_as_half(v)) : bf2f(v);
}

// Term `term` of eight FP32 values, as BF16 pairs.  An infinity or a NaN is the
// first term's alone.
__device__ __forceinline__ void terms_of(const float (&v)[8], int term, uint32_t (&b)[4]) {
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(v[i]);
    const bool finite = (u & 0x7F800000u) != 0x7F800000u;
    const float first = __uint_as_float(u & 0xFFFF0000u), left = v[i] - first;
    const float second = __uint_as_float(__float_as_uint(left) & 0xFFFF0000u);
    // (A NaN whose set bits are cut off would be an infinity.)
    if (term == 0) t[i] = v[i] != v[i] ? 0x7FC00000u : u & 0xFFFF0000u;
    else t[i] = finite ? __float_as_uint(term == 1 ? second : left - second) & 0xFFFF0000u : 0u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = t[2 * i] >> 16 | t[2 * i + 1];
}

// XK: 0 BF16, 1 FP16, 2 FP32 (TERMS columns a token).  MT row tiles of 16 to a
// warp (GATED: of gate and of up), NT column tiles of 8.  Eight warps share K.
template <int XK, int TERMS, int MT, int NT, bool GATED, int GROUP>
__global__ void __launch_bounds__(kWarps * 32) k_w4(const W4Args a) {
  constexpr bool BF = XK != 1;
  constexpr int ROWS = GATED ? 16 : 16 * MT;      // output features of a CTA
  constexpr int COLS = 8 * NT, TOK = COLS / TERMS;
  __shared__ float red[kWarps][16 * MT][COLS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane >> 2, t = lane & 3;
  const long long n0 = (long long)blockIdx.x * ROWS;
  const int t0 = blockIdx.y * TOK;
  const int tokens = min(TOK, a.T - t0), cols = tokens * TERMS;
  const long long K = a.w.K, N = a.w.N, runs = (K + kW4Run - 1) / kW4Run, pitch = runs * 64;
  const long long groups = (K + GROUP - 1) / GROUP;
  float sum[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) sum[i][j][c] = 0.0f;

  // Rows q and q + 8 of each row tile; past the last row the last again, not stored.
  const uint8_t* codes[MT][2];
  const void* scales[MT];
  long long row[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const W4Matrix& w = GATED && i == 1 ? a.w2 : a.w;
      row[i][h] = min(n0 + (GATED ? 0 : 16 * i) + q + 8 * h, N - 1);
      codes[i][h] = w.codes + row[i][h] * pitch + 16 * t;
      row[i][h] *= groups;
      scales[i] = w.scales;
    }
  constexpr int U = MT * NT >= 4 ? 2 : 4;   // runs whose codes are loaded at once
  grid_dep_wait();
  grid_dep_launch();
  for (long long b0 = warp; b0 < runs; b0 += U * kWarps) {
    uint4 code[U][MT][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          code[u][i][h] = b0 + u * kWarps < runs ? ld_stream(codes[i][h] + (b0 + u * kWarps) * 64) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long b = b0 + u * kWarps;
      if (b >= runs) break;
      float c[MT][NT][4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (g * 32 % GROUP == 0) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v) c[i][j][v] = 0.0f;
        }
        const long long k = b * kW4Run + g * 32 + t * 8;
        uint32_t xb[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int col = 8 * j + q;
          xb[j][0] = xb[j][1] = xb[j][2] = xb[j][3] = 0u;
          if (col < cols && k < K) {
            const long long at = (long long)(t0 + col / TERMS) * a.ldx + k;
            if constexpr (XK == 2) {
              const float* p = static_cast<const float*>(a.x) + at;
              float v[8];
              if (k + 8 <= K && ((uintptr_t)p & 15u) == 0) {
                Io<DETFFN_F32>::ld8(p, v);
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = k + e < K ? p[e] : 0.0f;
              }
              terms_of(v, col % TERMS, xb[j]);
            } else {
              const uint16_t* p = static_cast<const uint16_t*>(a.x) + at;
              if (k + 8 <= K && ((uintptr_t)p & 15u) == 0) {
                const uint4 v = *reinterpret_cast<const uint4*>(p);
                xb[j][0] = v.x, xb[j][1] = v.y, xb[j][2] = v.z, xb[j][3] = v.w;
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (k + e < K) xb[j][e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint32_t w0 = g == 0 ? code[u][i][0].x : g == 1 ? code[u][i][0].y : g == 2 ? code[u][i][0].z : code[u][i][0].w;
          const uint32_t w1 = g == 0 ? code[u][i][1].x : g == 1 ? code[u][i][1].y : g == 2 ? code[u][i][1].z : code[u][i][1].w;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t a0 = pair<BF>(w0, 2 * s), a1 = pair<BF>(w1, 2 * s), a2 = pair<BF>(w0, 2 * s + 1),
                           a3 = pair<BF>(w1, 2 * s + 1);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma<BF>(c[i][j], a0, a1, a2, a3, xb[j][2 * s], xb[j][2 * s + 1]);
          }
        }
        if ((g + 1) * 32 % GROUP == 0) {
          const long long at = (b * kW4Run + g * 32) / GROUP;
          if (at < groups) {   // (a group past the last column of K has no scale)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              const float s0 = ld_scale(scales[i], row[i][0] + at, a.w.stype), s1 = ld_scale(scales[i], row[i][1] + at, a.w.stype);
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                sum[i][j][0] = fmaf(s0, c[i][j][0], sum[i][j][0]);
                sum[i][j][1] = fmaf(s0, c[i][j][1], sum[i][j][1]);
                sum[i][j][2] = fmaf(s1, c[i][j][2], sum[i][j][2]);
                sum[i][j][3] = fmaf(s1, c[i][j][3], sum[i][j][3]);
              }
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[warp][16 * i + q + 8 * (v / 2)][8 * j + 2 * t + v % 2] = sum[i][j][v];
  __syncthreads();
  // The warps' sums in order, a token's terms from the smallest.
  for (int o = threadIdx.x; o < ROWS * tokens; o += kWarps * 32) {
    const int r = o % ROWS, tk = o / ROWS;
    float v[GATED ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (GATED ? 2 : 1); ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int e = TERMS - 1; e >= 0; --e) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += red[w][16 * i + r][tk * TERMS + e];
        v[i] += s;
      }
    }
    if (n0 + r >= N) continue;
    const float y = GATED ? v[0] * sigma<false>(v[0]).s * v[GATED ? 1 : 0] : v[0];
    const long long at = (t0 + tk) * a.ldo + n0 + r;
    if (a.otype == DETFFN_F32) static_cast<float*>(a.out)[at] = y;
    else if (a.otype == DETFFN_F16) Io<DETFFN_F16>::st(static_cast<uint16_t*>(a.out) + at, y);
    else Io<DETFFN_BF16>::st(static_cast<uint16_t*>(a.out) + at, y);
  }
}

template <int XK, int TERMS, int MT, int NT, bool GATED>
cudaError_t run_group(const W4Args& a, cudaStream_t st) {
  constexpr int ROWS = GATED ? 16 : 16 * MT, TOK = 8 * NT / TERMS;
  const dim3 grid((unsigned)((a.w.N + ROWS - 1) / ROWS), (unsigned)((a.T + TOK - 1) / TOK));
  if (a.w.group == 32) return launch_dependent(k_w4<XK, TERMS, MT, NT, GATED, 32>, grid, kWarps * 32, 0, st, a);
  if (a.w.group == 64) return launch_dependent(k_w4<XK, TERMS, MT, NT, GATED, 64>, grid, kWarps * 32, 0, st, a);
  return launch_dependent(k_w4<XK, TERMS, MT, NT, GATED, 128>, grid, kWarps * 32, 0, st, a);
}

template <int XK, int TERMS>
cudaError_t run(const W4Args& a, cudaStream_t st) {
  const int cols = a.T * TERMS;
  if (a.w2.codes) {
    if (cols <= 8) return run_group<XK, TERMS, 2, 1, true>(a, st);
    return run_group<XK, TERMS, 2, 2, true>(a, st);
  }
  if (cols <= 8) return run_group<XK, TERMS, 1, 1, false>(a, st);
  return run_group<XK, TERMS, 2, 2, false>(a, st);
}

// One warp takes runs of 128 weights of a row, four neighbours a lane.
template <int DT>
__global__ void __launch_bounds__(256) k_pack(const typename Io<DT>::E* w, long long ld, const W4Matrix m) {
  const int lane = threadIdx.x & 31;
  const long long runs = (m.K + kW4Run - 1) / kW4Run, groups = (m.K + m.group - 1) / m.group;
  grid_dep_wait();
  grid_dep_launch();
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < m.N * runs; i += 8ll * gridDim.x) {
    const long long n = i / runs, b = i - n * runs, k = b * kW4Run + 4 * lane;
    float v[4], top = 0.0f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = k + j < m.K ? Io<DT>::ld(w + n * ld + k + j) : 0.0f;
      top = fmaxf(top, fabsf(v[j]));
      bad |= !isfinite(v[j]);
    }
    for (int d = 1; 4 * d < m.group; d <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      bad |= __shfl_xor_sync(0xffffffffu, (int)bad, d) != 0;
    }
    float s = bad ? __int_as_float(0x7FC00000) : __fdiv_rn(top, 7.0f);
    if (m.stype == DETFFN_F16) s = __half2float(__float2half_rn(s));
    else if (m.stype == DETFFN_BF16) s = bf2f(f2bf(s));
    if (!isfinite(s)) s = __int_as_float(0x7FC00000);   // (also a scale that its type cannot hold)
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float c = s > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(v[j], s)), -7.0f), 7.0f) : 0.0f;
      word |= (uint32_t)((int)c + 8) << (4 * (j / 2 + 4 * (j % 2)));
    }
    // An even lane holds codes 0 .. 3 of its word, the next one codes 4 .. 7, two nibbles on.
    word <<= 8 * (lane & 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    if ((lane & 1) == 0)
      reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(m.codes) + i * 64)[(lane % 8) / 2 * 4 + lane / 8] = word;
    if (4 * lane % m.group == 0 && k < m.K) {
      const long long at = n * groups + k / m.group;
      void* to = const_cast<void*>(m.scales);
      if (m.stype == DETFFN_F32) static_cast<float*>(to)[at] = s;
      else if (m.stype == DETFFN_F16) Io<DETFFN_F16>::st(static_cast<uint16_t*>(to) + at, s);
      else Io<DETFFN_BF16>::st(static_cast<uint16_t*>(to) + at, s);
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(256) k_unpack(const W4Matrix m, typename Io<DT>::E* w, long long ld) {
  const int lane = threadIdx.x & 31;
  const long long runs = (m.K + kW4Run - 1) / kW4Run, groups = (m.K + m.group - 1) / m.group;
  grid_dep_wait();
  grid_dep_launch();
  for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < m.N * runs; i += 8ll * gridDim.x) {
    const long long n = i / runs, b = i - n * runs, k = b * kW4Run + 4 * lane;
    const uint32_t word = reinterpret_cast<const uint32_t*>(m.codes + i * 64)[(lane % 8) / 2 * 4 + lane / 8] >> (8 * (lane & 1));
    if (k >= m.K) continue;
    const float s = ld_scale(m.scales, n * groups + k / m.group, m.stype);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k + j < m.K) Io<DT>::st(w + n * ld + k + j, s * (float)((int)(word >> (4 * (j / 2 + 4 * (j % 2))) & 15u) - 8));
  }
}

unsigned pack_grid(const W4Matrix& m, int sm_count) {
  const long long want = (m.N * ((m.K + kW4Run - 1) / kW4Run) + 7) / 8, most = 8ll * sm_count;
  return (unsigned)(want < most ? want : most);
}

}  // namespace

cudaError_t launch_w4_matvec(const W4Args& a, int, cudaStream_t st) {
  if (a.xtype == DETFFN_BF16) return run<0, 1>(a, st);
  if (a.xtype == DETFFN_F16) return run<1, 1>(a, st);
  return a.terms == 2 ? run<2, 2>(a, st) : run<2, 3>(a, st);
}

cudaError_t launch_w4_pack(const void* w, long long ld, int dtype, const W4Matrix& to, int sm_count, cudaStream_t st) {
  const dim3 grid(pack_grid(to, sm_count));
  if (dtype == DETFFN_F32) return launch_dependent(k_pack<DETFFN_F32>, grid, 256, 0, st, static_cast<const float*>(w), ld, to);
  const uint16_t* p = static_cast<const uint16_t*>(w);
  return dtype == DETFFN_F16 ? launch_dependent(k_pack<DETFFN_F16>, grid, 256, 0, st, p, ld, to)
                             : launch_dependent(k_pack<DETFFN_BF16>, grid, 256, 0, st, p, ld, to);
}

cudaError_t launch_w4_unpack(const W4Matrix& from, void* w, long long ld, int dtype, int sm_count, cudaStream_t st) {
  const dim3 grid(pack_grid(from, sm_count));
  if (dtype == DETFFN_F32) return launch_dependent(k_unpack<DETFFN_F32>, grid, 256, 0, st, from, static_cast<float*>(w), ld);
  uint16_t* p = static_cast<uint16_t*>(w);
  return dtype == DETFFN_F16 ? launch_dependent(k_unpack<DETFFN_F16>, grid, 256, 0, st, from, p, ld)
                             : launch_dependent(k_unpack<DETFFN_BF16>, grid, 256, 0, st, from, p, ld);
}

}  // namespace detffn
