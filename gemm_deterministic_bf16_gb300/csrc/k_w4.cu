// k_w4.cu -- products of a few tokens with matrices of 4-bit codes and a scale
// for each group of 32, 64 or 128 codes of a row.
//
//   y[t, n] = sum over groups g of  s[n, g] * ( sum over k in g of (code[n, k] - 8) * x[t, k] )
//
// What has to be moved is the weights' bytes (half a byte a weight and the scales).
// At the copy rate (6.68 TB/s to 152 SMs of 2070 MHz) an SM takes in some 41 weights a
// cycle, so
// the arithmetic goes to the tensor cores by mma.sync m16n8k16, straight from
// registers: the weights are the 16-row operand, eight columns (tokens,
// or the terms of their activations) the other, and a weight is read and
// converted once for all columns of a pass (8, 16 or 32).  A code becomes BF16 or FP16 by putting its
// bits into the mantissa of 128 or 1024 and subtracting 136 or 1032: exact, as
// are all products with a 16-bit x.  A group's sum is one accumulation in FP32,
// scaled and added to the row's FP32 sum.
//
// An FP32 activation is three BF16 terms (together all 24 bits), in columns of
// their own; a small kernel lays them out first, and rows that are not on
// 16-byte boundaries.  The hidden activation of the gated FFN goes from one
// launch to the next as two terms (16 bits), three for FP32: two are off by at most
// 2^-16 of a value, which a result of 8 or 11 bits does not show (the FFN of one token, H
// = 4096, I = 12288, BF16, is 1.67666e-3 of its norm from the 64-bit one, with h in FP32
// 1.67665e-3), and a third would be half as many columns again.
//
// The order of the codes makes this a matter of plain vectors: lane 4 r + t of
// a warp holds row r (and r + 8) of the 16-row operand and columns 2 t, 2 t + 1,
// 2 t + 8, 2 t + 9 of each 16 of K.  As any order of K serves, chunk t of a run
// of 128 codes (16 bytes) holds what lane t needs of it: word g the codes 32 g +
// 8 t .. + 7 of group quarter g, nibble p of it code 2 (p mod 4) + p / 4, so
// that a mask and a shift leave neighbours in the two halves of a register.
//
// Converting 2048 weights takes a warp some 90 instructions besides the loads,
// half of what an SM can issue in the time their bytes take; so the loop has little
// else.  Codes and scales come by cp.async, each lane's own pieces an item ahead in a
// ring of shared memory that outlasts the row tiles, x from L1 without tests.
//
// It reaches 41 to 61 % of the copy rate: 8 tokens of a 131072 x 4096 matrix in FP16,
// groups of 64, 78 us (floor 43); the FFN of one token, H = 4096, I = 12288, BF16, groups of
// 128, 26.6 us (floor 11.6); one token through 4096 x 4096 4.7 us (floor 1.3).  A run of
// 128 codes of 16 rows takes 190 to 210 instructions, of which the integer pipe, which
// issues one in two cycles, has 72 to 83; but issue is at 47 to 61 % and HBM at 26 to 45, so
// nothing is full: the up to 24 warps an SM that registers and rings leave room for do
// not cover the latency.  With more columns it is latency too: in the
// FFN of 32 tokens (70 us; 22 of them the matrix instructions', one in two cycles for an
// SM) eight warps an SM, all that the sums leave registers for, issue in 31 % of the
// cycles and wait for results of a fixed latency most, then for x from L2; 2.5 tiles
// an SM and 128 CTAs leave a sixth of it idle.  Neither sixteen warps that share x in
// shared memory (92 us), nor x in each warp's ring (96), nor four by two tiles with two
// CTAs an SM (93) does better: all three add more instructions than they hide.
#include <stddef.h>

#include <type_traits>

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

// The same with nothing to add to.
template <bool BF16>
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}

// The four pairs of codes 2 i and 2 i + 1 of a word, less 8, in the halves of a
// register: 128 + code - 136 in BF16; 1024 + code - 1032, or (1024 + 16 code) / 16 -
// 72 without a shift, in FP16.  All exact.
template <bool BF16>
__device__ __forceinline__ void pairs_of(uint32_t word, uint32_t (&r)[4]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(and_or(word >> (4 * i), 0x000F000Fu, 0x43004300u)), "r"(0x3F803F80u), "r"(0xC308C308u));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? word : word >> 8;
      if (i % 2 == 0) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(and_or(w, 0x000F000Fu, 0x64006400u)), "r"(0x3C003C00u), "r"(0xE408E408u));
      else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(and_or(w, 0x00F000F0u, 0x64006400u)), "r"(0x2C002C00u), "r"(0xD480D480u));
    }
  }
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// The first n of four bytes, zeros behind.
__device__ __forceinline__ void copy4(uint32_t to, const void* from, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float ld_scale(const void* p, long long i, int type) {
  if (type == DETFFN_F32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t v = __ldg(static_cast<const uint16_t*>(p) + i);
  return type == DETFFN_F16 ? __half2float(__ushort_as_half(v)) : bf2f(v);
}

// Terms of an FP32 value: the leading eight bits of what the ones before left,
// the last one rounded.  An infinity or a NaN is the first term's alone.
__device__ __forceinline__ void terms_of(float v, int n, uint16_t (&t)[3]) {
  const uint32_t u = __float_as_uint(v);
  t[1] = t[2] = 0;
  if ((u & 0x7F800000u) == 0x7F800000u) {
    t[0] = v != v ? 0x7FC0u : (uint16_t)(u >> 16);   // (a NaN's set bits may be the low ones)
    return;
  }
  t[0] = (uint16_t)(u >> 16);
  const float left = v - bf2f(t[0]);
  t[1] = n == 2 ? f2bf(left) : (uint16_t)(__float_as_uint(left) >> 16);
  if (n == 3) t[2] = f2bf(left - bf2f(t[1]));
}

// Runs of an item (of one row and column tile two, which halve what a run costs
// besides its conversion), and items of a warp's ring: one is used while the
// other is on its way.  More would leave the activations no room in L1.
template <int MT, int NT> constexpr int kRuns = MT * NT == 1 ? 2 : 1;
template <int MT, int NT> constexpr int kRing = 2;

// Shared memory of a warp's ring item: codes [row half][lane], then scales [row][4 words].
template <int MT, int NT> struct Item {
  uint4 code[kRuns<MT, NT>][2 * MT][32];
  uint32_t scale[kRuns<MT, NT>][16 * MT][4];
};
template <int MT, int NT> struct Smem {
  static constexpr int kRed = MT < 4 ? 2 : 1;
  Item<MT, NT> ring[kWarps][kRing<MT, NT>];
  float red[kRed][kWarps][16 * MT][8 * NT + 1];
};

// MT row tiles of 16 to a warp (GATED: half of gate, half of up), NT column
// tiles of 8.  The eight warps share K, a run of 128 each in turn.
template <bool BF, int MT, int NT, bool GATED, int GROUP>
__global__ void __launch_bounds__(kWarps * 32, MT * NT <= 2 ? 3 : MT * NT <= 4 ? 2 : 1) k_w4(const W4Args a) {
  constexpr int ROWS = GATED ? 8 * MT : 16 * MT;  // output features of a tile
  constexpr int PER = kW4Run / GROUP;             // groups of a run
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<MT, NT>& sm = *reinterpret_cast<Smem<MT, NT>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane >> 2, t = lane & 3;
  const int terms = a.x.terms, tok = 8 * NT / terms, t0 = blockIdx.y * tok, tokens = min(tok, a.T - t0), cols = tokens * terms;
  const int N = (int)a.w.N, K = (int)a.w.K, runs = (K + kW4Run - 1) / kW4Run, groups = (K + GROUP - 1) / GROUP;
  const int tiles = (N + ROWS - 1) / ROWS, Kx = (K + 7) & ~7;
  const bool wide = a.w.stype == DETFFN_F32;
  // Words of scales of a run that a lane copies: word t of its rows; a run's
  // first scale of 16 bits may be the upper half of its word.
  const int words = wide ? PER : PER / 2 + 1, es = wide ? 4 : 2;
  const long long row_scales = (long long)groups * es;

  // Columns past the last read the last one's x; their sums are not used.
  const uint16_t* x[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int col = min(8 * j + q, cols - 1);
    x[j] = static_cast<const uint16_t*>(a.x.p) + (col % terms) * a.x.plane + (long long)(t0 + col / terms) * a.x.ld + 8 * t +
           warp * kW4Run;
  }

  // The matrix, and the row of it, of row q + 8 h of row tile i; past the last row the last again, not stored.
  auto matrix_of = [&](int i) -> const W4Matrix& { return GATED && i >= MT / 2 ? a.w2 : a.w; };
  auto row_of = [&](int tile, int i, int h) {
    return min(tile * ROWS + 16 * (GATED && i >= MT / 2 ? i - MT / 2 : i) + q + 8 * h, N - 1);
  };
  // The next copies: pointers of rows q, distances to rows q + 8 (both in a tile).
  const uint8_t* code_at[MT];
  const char* scale_at[MT];
  uint32_t code_8[MT], scale_8[MT];
  bool inside = false;   // the words of the tile's scales all lie in the array (a run's may reach 16 bytes past its row)
  auto aim = [&](int tile) {
    inside = (N - (tile + 1ll) * ROWS) * row_scales >= 16;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const long long r = row_of(tile, i, 0), r8 = row_of(tile, i, 1);
      code_at[i] = matrix_of(i).codes + (r * runs + warp) * 64 + 16 * t;
      code_8[i] = (uint32_t)(r8 - r) * (uint32_t)runs * 64;
      const char* s = static_cast<const char*>(matrix_of(i).scales) + 4 * t;
      const long long at = (r * row_scales + warp * PER * es) & ~3ll, at8 = (r8 * row_scales + warp * PER * es) & ~3ll;
      scale_at[i] = s + at;
      scale_8[i] = (uint32_t)(at8 - at);
    }
  };
  using It = Item<MT, NT>;
  constexpr uint32_t ITEM = sizeof(It);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(&sm.ring[warp][0]), lane_code = lane * 16,
                 lane_scale = (uint32_t)offsetof(It, scale) + q * 16 + 4 * t;
  uint32_t put = ring;
  int ntile = blockIdx.x, nrun = warp;
  if (warp >= runs) ntile = tiles;   // (no run for this warp)
  auto copy_run = [&](auto run_of_item) {
    constexpr int u = decltype(run_of_item)::value;
    const uint32_t code_to = put + lane_code + u * MT * 1024, scale_to = put + lane_scale + u * MT * 256;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      copy16(code_to + i * 1024, code_at[i] + u * kWarps * 64);
      copy16(code_to + i * 1024 + 512, code_at[i] + code_8[i] + u * kWarps * 64);
    }
    if (t >= words) return;
    const int step = u * kWarps * PER * es;
    if (inside) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        copy4(scale_to + i * 256, scale_at[i] + step);
        copy4(scale_to + i * 256 + 128, scale_at[i] + scale_8[i] + step);
      }
    } else {   // (the array's end: two bytes of a word, or none)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const char* base = static_cast<const char*>(matrix_of(i).scales);
          const char* from = scale_at[i] + (h ? scale_8[i] : 0) + step;
          const long long left = (long long)N * row_scales - (from - base);
          copy4(scale_to + i * 256 + h * 128, left > 0 ? from : base, (int)min(max(left, 0ll), 4ll));
        }
    }
  };
  auto copy_next = [&]() {
    if (ntile < tiles) {
      copy_run(std::integral_constant<int, 0>());
      if (kRuns<MT, NT> == 2 && nrun + kWarps < runs) copy_run(std::integral_constant<int, kRuns<MT, NT> - 1>());
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        code_at[i] += kRuns<MT, NT> * kWarps * 64;
        scale_at[i] += kRuns<MT, NT> * kWarps * PER * es;
      }
      nrun += kRuns<MT, NT> * kWarps;
      if (nrun >= runs) {
        nrun = warp;
        ntile += gridDim.x;
        if (ntile < tiles) aim(ntile);
      }
    }
    copies_commit();
    put += ITEM;
    if (put == ring + kRing<MT, NT> * ITEM) put = ring;
  };

  if (ntile < tiles) {
    aim(ntile);
    // The first codes on their way to L2 (where nothing the launch before may write can go stale).
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(code_at[i]));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(code_at[i] + code_8[i]));
    }
  }
  grid_dep_wait();
  grid_dep_launch();
#pragma unroll
  for (int i = 0; i < kRing<MT, NT> - 1; ++i) copy_next();

  int use = 0, buf = 0;
  const int full = Kx / kW4Run;   // whole runs
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    float sum[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[i][j][v] = 0.0f;
    int half[MT][2];   // 16, where the runs' first scale is the upper half of its word
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) half[i][h] = ((row_of(tile, i, h) & groups) + warp * PER & 1) * 16;
    const uint16_t* xr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xr[j] = x[j];
    // Run u of an item; LAST: the one that K ends in.
    auto one_run = [&](auto last, auto run_of_item, int run) {
      constexpr bool LAST = decltype(last)::value;
      constexpr int u = decltype(run_of_item)::value;
      uint4 xv[4][NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4* p = reinterpret_cast<const uint4*>(xr[j] + u * kWarps * kW4Run);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if constexpr (LAST) {
            xv[g][j] = make_uint4(0, 0, 0, 0);
            if (run * kW4Run + 32 * g + 8 * t < Kx) xv[g][j] = p[4 * g];
          } else {
            xv[g][j] = p[4 * g];
          }
        }
      }
      if constexpr (u == 0) {
        __syncwarp();   // (all lanes are done with the item that is written next)
        copy_next();
        copies_wait<kRing<MT, NT> - 1>();
        __syncwarp();   // (scales are copied for neighbours too)
      }
      const It& it = sm.ring[warp][use];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint4 c0 = it.code[u][2 * i][lane], c1 = it.code[u][2 * i + 1][lane];
        float s[2][PER];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t* ws = it.scale[u][16 * i + 8 * h + q];
          if (wide) {
#pragma unroll
            for (int n = 0; n < PER; ++n) s[h][n] = __uint_as_float(ws[n]);
          } else {
            uint32_t v[(PER + 1) / 2];
#pragma unroll
            for (int n = 0; n < (PER + 1) / 2; ++n)
              v[n] = PER == 1 ? ws[0] >> half[i][h] : __funnelshift_r(ws[n], ws[n + 1], half[i][h]);
#pragma unroll
            for (int n = 0; n < PER; ++n) {
              if (a.w.stype == DETFFN_F16) s[h][n] = __half2float(__ushort_as_half((uint16_t)(v[n / 2] >> (n % 2 * 16))));
              else s[h][n] = __uint_as_float(n % 2 ? v[n / 2] & 0xFFFF0000u : v[n / 2] << 16);
            }
          }
          if constexpr (LAST) {   // (a group past the last column of K has no scale)
#pragma unroll
            for (int n = 0; n < PER; ++n)
              if (run * PER + n >= groups) s[h][n] = 0.0f;
          }
        }
        float c[NT][4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t w0 = g == 0 ? c0.x : g == 1 ? c0.y : g == 2 ? c0.z : c0.w;
          const uint32_t w1 = g == 0 ? c1.x : g == 1 ? c1.y : g == 2 ? c1.z : c1.w;
          uint32_t p0[4], p1[4];
          pairs_of<BF>(w0, p0);
          pairs_of<BF>(w1, p1);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (g * 32 % GROUP == 0) mma_first<BF>(c[j], p0[0], p1[0], p0[1], p1[1], xv[g][j].x, xv[g][j].y);
            else mma<BF>(c[j], p0[0], p1[0], p0[1], p1[1], xv[g][j].x, xv[g][j].y);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) mma<BF>(c[j], p0[2], p1[2], p0[3], p1[3], xv[g][j].z, xv[g][j].w);
          if ((g + 1) * 32 % GROUP == 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int v = 0; v < 4; ++v) sum[i][j][v] = fmaf(s[v / 2][g * 32 / GROUP], c[j][v], sum[i][j][v]);
          }
        }
      }
    };
    auto next_item = [&]() {
      if (++use == kRing<MT, NT>) use = 0;
#pragma unroll
      for (int j = 0; j < NT; ++j) xr[j] += kRuns<MT, NT> * kWarps * kW4Run;
    };
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, kRuns<MT, NT> - 1>;
    int run = warp;
#pragma unroll 1
    for (; run + (kRuns<MT, NT> - 1) * kWarps < full; run += kRuns<MT, NT> * kWarps) {
      one_run(std::false_type(), First(), run);
      if constexpr (kRuns<MT, NT> == 2) one_run(std::false_type(), Second(), run + kWarps);
      next_item();
    }
    // What is left: a run with none or the last behind it, or the last.
    if (run < runs) {
      if (kRuns<MT, NT> == 2 && run < full) {
        one_run(std::false_type(), First(), run);
        if (run + kWarps < runs) one_run(std::true_type(), Second(), run + kWarps);
      } else {
        one_run(std::true_type(), First(), run);
      }
      next_item();
    }
    float (&red)[kWarps][16 * MT][8 * NT + 1] = sm.red[Smem<MT, NT>::kRed == 2 ? buf : 0];
    if (Smem<MT, NT>::kRed == 1) __syncthreads();   // (the last tile's readers)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[warp][16 * i + q + 8 * (v / 2)][8 * j + 2 * t + v % 2] = sum[i][j][v];
    __syncthreads();   // (with two buffers one a tile: the other's readers are past it when it is written again)
    // The warps' sums in order, a token's terms from the smallest.
    for (int o = threadIdx.x; o < ROWS * tokens; o += kWarps * 32) {
      const int r = o % ROWS, tk = o / ROWS, n = tile * ROWS + r;
      float v[2];
#pragma unroll
      for (int i = 0; i < (GATED ? 2 : 1); ++i) {
        v[i] = 0.0f;
        for (int e = terms - 1; e >= 0; --e) {
          float s = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) s += red[w][ROWS * i + r][tk * terms + e];
          v[i] += s;
        }
      }
      if (n >= (GATED ? (N + 7) & ~7 : N)) continue;
      const long long at = (t0 + tk) * a.ldo + n;
      if constexpr (GATED) {
        uint16_t h[3];
        terms_of(n < N ? v[0] * sigma<false>(v[0]).s * v[1] : 0.0f, a.terms, h);   // (zeros to a multiple of 8)
        for (int e = 0; e < a.terms; ++e) static_cast<uint16_t*>(a.out)[at + e * a.plane] = h[e];
      } else if (a.otype == DETFFN_F32) {
        static_cast<float*>(a.out)[at] = v[0];
      } else {
        static_cast<uint16_t*>(a.out)[at] = a.otype == DETFFN_F16 ? __half_as_ushort(__float2half_rn(v[0])) : f2bf(v[0]);
      }
    }
  }
}

template <bool BF, int MT, int NT, bool GATED, int GROUP>
cudaError_t run_one(const W4Args& a, int sm_count, cudaStream_t st) {
  constexpr int ROWS = GATED ? 8 * MT : 16 * MT, SM = MT * NT <= 2 ? 3 : MT * NT <= 4 ? 2 : 1;
  // Where one or two tiles an SM are all there are, more shared memory than is used
  // keeps more CTAs than that from one SM while others have fewer (N = 4096, K = 12288,
  // one token: 12.1 and 9.5 us).
  constexpr int kAlone = 120 * 1024, kTwo = 80 * 1024, kUsed = (int)sizeof(Smem<MT, NT>);
  static PerDevice ready;
  const cudaError_t e = once_per_device(ready, [] {
    return cudaFuncSetAttribute(k_w4<BF, MT, NT, GATED, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kUsed > kAlone ? kUsed : kAlone);
  });
  if (e != cudaSuccess) return e;
  const int tok = 8 * NT / a.x.terms, passes = (a.T + tok - 1) / tok;
  const long long tiles = (a.w.N + ROWS - 1) / ROWS, slots = (long long)SM * sm_count, ctas = (tiles < slots ? tiles : slots) * passes;
  const int least = ctas <= sm_count ? kAlone : ctas <= 2ll * sm_count ? kTwo : 0;
  return launch_dependent(k_w4<BF, MT, NT, GATED, GROUP>, dim3((unsigned)(tiles < slots ? tiles : slots), (unsigned)passes),
                          kWarps * 32, kUsed > least ? kUsed : least, st, a);
}
template <bool BF, int MT, int NT, bool GATED>
cudaError_t run_group(const W4Args& a, int sm_count, cudaStream_t st) {
  if (a.w.group == 32) return run_one<BF, MT, NT, GATED, 32>(a, sm_count, st);
  if (a.w.group == 64) return run_one<BF, MT, NT, GATED, 64>(a, sm_count, st);
  return run_one<BF, MT, NT, GATED, 128>(a, sm_count, st);
}
// Columns in passes of 8, 16 or 32, weights read again for each: the CTAs of a pass
// follow those of the last, so from L2 where the matrix fits it, else from HBM.  Four
// row and column tiles read x from L1 half as often as two, and leave an SM eight
// warps instead of sixteen: they pay for gate and up from 17 columns on (FFN of 8
// tokens in FP32, H = 4096, I = 12288: 59 and 55 us), else from 33 (16 tokens in BF16: 52 and
// 41.5 us with two tiles; 32 tokens, 64 columns: 70.6 and 74.6).
template <bool BF>
cudaError_t run(const W4Args& a, int sm_count, cudaStream_t st) {
  const int cols = a.T * a.x.terms;
  if (a.w2.codes) {
    if (cols <= 8) return run_group<BF, 2, 1, true>(a, sm_count, st);
    if (cols <= 16) return run_group<BF, 2, 2, true>(a, sm_count, st);
    return run_group<BF, 4, 4, true>(a, sm_count, st);
  }
  if (cols <= 8) return run_group<BF, 1, 1, false>(a, sm_count, st);
  if (cols <= 32) return run_group<BF, 2, 2, false>(a, sm_count, st);
  return run_group<BF, 4, 4, false>(a, sm_count, st);
}

// Rows as 16-bit terms, K padded with zeros to a multiple of 8.
template <int DT>
__global__ void __launch_bounds__(256) k_rows(const typename Io<DT>::E* x, long long ldx, long long T, long long K, int terms,
                                              uint16_t* to) {
  const long long Kp = w4_pad(K), n = T * Kp;
  grid_dep_wait();
  grid_dep_launch();
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += 256ll * gridDim.x) {
    const long long r = i / Kp, k = i - r * Kp;
    if constexpr (DT == DETFFN_F32) {
      uint16_t h[3] = {0, 0, 0};
      if (k < K) terms_of(x[r * ldx + k], terms, h);
      for (int e = 0; e < terms; ++e) to[i + e * n] = h[e];
    } else {
      to[i] = k < K ? x[r * ldx + k] : (uint16_t)0;
    }
  }
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

cudaError_t launch_w4_rows(const void* x, long long ldx, int dtype, long long T, long long K, int terms, void* to,
                           int sm_count, cudaStream_t st) {
  const long long want = (T * w4_pad(K) + 255) / 256, most = 4ll * sm_count;
  const dim3 grid((unsigned)(want < most ? want : most));
  uint16_t* p = static_cast<uint16_t*>(to);
  if (dtype == DETFFN_F32) return launch_dependent(k_rows<DETFFN_F32>, grid, 256, 0, st, static_cast<const float*>(x), ldx, T, K, terms, p);
  return launch_dependent(k_rows<DETFFN_BF16>, grid, 256, 0, st, static_cast<const uint16_t*>(x), ldx, T, K, terms, p);
}

cudaError_t launch_w4_matvec(const W4Args& a, int sm_count, cudaStream_t st) {
  return a.x.f16 ? run<false>(a, sm_count, st) : run<true>(a, sm_count, st);
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
