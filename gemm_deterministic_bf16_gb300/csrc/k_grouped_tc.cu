// k_grouped_tc.cu -- matrix products grouped by expert on the tensor cores, BF16
// and FP16 (the formulas are those of k_grouped.cu).
//
// Persistent pairs of CTAs (cta_group::2), one pair on two SMs, take output
// tiles of 256 features x up to 256 rows in turn:
//
//            MMA rows (256)          MMA columns (up to 256)   contraction
//   out      features n of W[e]      rows of x                 K
//   dx       features k of W[e]      rows of dout              N
//   dW       features k of x         features n of dout        rows of the expert
//
// so that the 32 lanes of a warp hold neighbours of one output row, and the
// ragged side, the rows of an expert, is the one whose size an MMA can choose
// (in steps of 32): an expert's rows are cut into equal tiles, and a tile's
// MMAs cover its rows, not 256.  Operands that run across the contraction in
// memory (W for dx, x and dout for dW) are read MN-major, without a copy.
//
// Each CTA of a pair loads its 128 rows of A and half of B by TMA, 128 of the
// contraction to a stage, counted by barriers of the first CTA, which issues the
// MMAs of both; FP32 sums in two halves of tensor memory, so that the next
// tile's MMAs run while four warps of each CTA (eight, where
// contractions are short) write the last one out.
//
// For dW the contraction ends with the expert's rows: those that the last 16 of
// it take in beyond are another expert's and are cleared in shared memory, in
// both operands (0 times an infinity is a NaN), by a warp that the last stage of
// a tile goes through.
//
// The experts' rows are read on the device.  Every pair works out all tiles
// from them and takes every (number of pairs)-th; the cut of the rows (the
// widest tile) is the one whose rounds of tiles, each at the cost of its widest
// tile, take least.
//
// What bounds it: at the MMA's full rate an SM takes in 64 bytes a cycle from L2, and
// its shared memory is read and written by 128.  A stage holds 128 of the contraction,
// as a wait and a commit for every 64 cost the issuing thread what their MMAs take.
// More stages in flight, and prefetches into L2 ahead of them, gain nothing or cost
// half the rate.  (Rows that two pairs share are loaded by each, not by multicast:
// the library also serves programs on several GPUs.  That was no faster: 315 us for
// 16384 x 4096 x 4096, 298 as it is.)
//
// BF16, 16384 x 4096 x 4096: 298 us forward, 300 dx, 347 dW (97, 97 and 83 % of the
// measured matrix rate); 16384 uneven rows of 16 experts, K = 4096, N = 1536: 151 to 155 us
// forward, 312 to 352 both gradients, by the power there is (70 to 72 and 62 to 70 %: six
// rounds of tiles on 76 pairs, the last in part empty); 99 rows of 64 experts, K = 2048, N
// = 768: 34.5 to 38.7 us (66 to 59 % of the copy rate); 1499 rows of 16 experts, K = 1416, N
// = 4096, FP16: 123 us (both gradients; 48 % of the copy rate: two rounds for dx, the
// results' way out for dW).
#include "elt.cuh"
#include "grouped.h"
#include "ptx.cuh"
#include "tc.h"

namespace detffn {
namespace {

constexpr int kThreads = 256;       // warp 0 loads, 1 issues MMAs, 2 clears, 3 cuts the rows into tiles, 4-7 write out
constexpr int kMostThreads = 384;   // and 8-11 too
constexpr int kStages = 3;
constexpr int kHalf = 128 * 128;    // bytes of an operand's part of a slice of 64 of the contraction
constexpr int kSlice = 2 * kHalf;
constexpr int kStep = 128;          // of the contraction to a stage: two slices
constexpr int kStage = 2 * kSlice;
constexpr int kCols = 256;          // columns of tensor memory to a tile's sums
constexpr int kChunk = 32;          // output rows that are staged at once
constexpr int kPitch = 256 + 16;    // of a staged row of 128 features: eight rows of a transposed store meet no bank twice
constexpr int kOutBytes = 2 * kChunk * kPitch;   // for each four warps that write out, kChunk rows
constexpr int kSuper = 8;           // feature tiles that are taken together

struct Bars {
  uint64_t full[kStages];    // first CTA: both CTAs' copies have landed
  uint64_t empty[kStages];   // both: the stage's MMAs are done
  uint64_t tail[kStages];    // both: this CTA's copies of a stage that is to be cleared have landed
  uint64_t accf[2];          // both: a tile's sums are done
  uint64_t acce[2];          // first CTA: both CTAs have read them
  uint64_t fin;
  uint32_t tmem;
  int abort, cap, total;
  int stopped;               // a timeout was recorded before this launch
};

struct Args {
  int what;                  // 0 out, 1 dx, 2 dW
  int E;
  long long R;               // rows of all experts
  const int* off;
  int F;                     // output features (MMA rows' side)
  int C;                     // contraction (out, dx)
  int N;                     // dW: output rows
  uint16_t* out;
  long long ldo, stride;     // row stride; dW: elements of a matrix
  int* status;
  long long spin;
  int stall;
  int sets;                  // of four warps that write out: 1 or 2
  int vec;                   // output rows lie on 16-byte boundaries
};

// First row, rows, and the tiles before each expert's.
struct Tables {
  int *beg, *cnt, *pre;
};
__host__ __device__ inline int tables_bytes(int E) { return ((3 * E + 1) * 4 + 15) & ~15; }
__device__ __forceinline__ Tables tables_at(unsigned char* p, int E) {
  Tables t;
  t.beg = reinterpret_cast<int*>(p);
  t.cnt = t.beg + E;
  t.pre = t.cnt + E;
  return t;
}

struct Tile {
  int e, f0;        // expert, first feature
  int r0, rows;     // first output row (of the expert; of dW[e]), output rows
  int nt;           // MMA columns: the rows in whole 32s
  int steps;        // stages of the contraction
  int last;         // positions of the last one
};

__device__ __forceinline__ int up32(int n) { return (n + 31) & ~31; }

__device__ __forceinline__ int feature_tiles(const Args& g) { return (g.F + 255) / 256; }

// l / d by m = (2^32 - 1) / d, for l < 2^31: the estimate is at most one short.
__device__ __forceinline__ int quotient(int l, int d, uint32_t m) {
  const int q = (int)__umulhi((uint32_t)l, m);
  return l - q * d >= d ? q + 1 : q;
}

// The tiles of a pair in order.  What a tile's
// place needs of divisions is kept for the expert, as all roles wait for it (dW of 16
// experts of 94 rows, K = 1416, N = 4096: 64 us with divisions, 60 without).
struct Walk {
  int e = -1, next = 0;                 // expert; the first tile of the one after it
  int first = 0, n = 0, wide = 0, steps = 0, last = 0;
  int area = 1, full, left;             // tiles of kSuper features; whole ones of them, features of the last
  uint32_t by_area = 0, by_left;
  __device__ __forceinline__ explicit Walk(const Args& g) {
    const int ft = feature_tiles(g);
    full = ft / kSuper;
    left = ft % kSuper;
    by_left = 0xFFFFFFFFu / (uint32_t)max(left, 1);
  }
  __device__ __forceinline__ Tile at(int id, const Args& g, const Tables& t, int cap) {
    if (id >= next) {
      do ++e;
      while (id >= t.pre[e + 1]);
      next = t.pre[e + 1];
      first = t.pre[e];
      n = g.what == 2 ? g.N : t.cnt[e];
      const int rt = (n + cap - 1) / cap, c = g.what == 2 ? t.cnt[e] : g.C;
      wide = up32(n / rt + (n % rt != 0));   // (at most cap, so the last tile has rows)
      steps = (c + kStep - 1) / kStep;
      last = c - (steps - 1) * kStep;
      area = rt * kSuper;
      by_area = 0xFFFFFFFFu / (uint32_t)area;
    }
    const int l = id - first, sb = quotient(l, area, by_area), m = l - sb * area;
    const int r = sb < full ? m / kSuper : quotient(m, left, by_left), c = m - r * (sb < full ? kSuper : left);
    Tile q;
    q.e = e;
    q.f0 = (sb * kSuper + c) * 256;
    q.r0 = r * wide;
    q.rows = min(wide, n - q.r0);
    q.nt = up32(q.rows);
    q.steps = steps;
    q.last = last;
    return q;
  }
};

// Four of the warps that write out (set 0 or 1).
__device__ __forceinline__ void out_sync(int set) { asm volatile("bar.sync %0, 128;" ::"r"(set + 1) : "memory"); }
// The same barrier; whether `ok` held in all 128 threads.
__device__ __forceinline__ bool out_all(int set, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.and.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(set + 1), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

struct Abort {
  int* mine;
  int* status;
  long long limit;
};
// (All lanes together.  REMOTE: what the other CTA's threads wrote before they
// arrived is seen after it.)
template <bool REMOTE = false>
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, const Abort& a) {
  bool ok = false, timeout = true;
  for (long long i = 0; i < a.limit; ++i) {
    if (REMOTE ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) {
      ok = true;
      timeout = false;
      break;
    }
    if ((i & 1023) == 1023 && *(volatile int*)a.mine) {
      timeout = false;
      break;
    }
  }
  if (timeout) {
    for (int c = 0; c < 2; ++c) cluster_st(cluster_addr(a.mine, c), 1);
    if (a.status) atomicExch(a.status, (int)DETFFN_ERR_TIMEOUT);
  }
  return __all_sync(0xffffffffu, ok) != 0;
}

template <int DT>
__global__ void __launch_bounds__(kMostThreads, 1)
    k_grouped_tc(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                 const __grid_constant__ CUtensorMap mB64, const __grid_constant__ CUtensorMap mB32,
                 const __grid_constant__ Args g) {
  extern __shared__ unsigned char raw[];
  // (The same offset in both CTAs: dynamic shared memory starts at the same address in each.)
  unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  unsigned char* staged = smem + kStages * kStage;
  Bars* bars = reinterpret_cast<Bars*>(staged + kOutBytes);
  const Tables t = tables_at(reinterpret_cast<unsigned char*>(bars) + ((sizeof(Bars) + 127) & ~127), g.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = (int)blockIdx.x / 2, pairs = (int)gridDim.x / 2;
  const Abort ab{&bars->abort, g.status, g.spin > 0 ? g.spin : kDefaultSpin};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 2);
      mbar_init(&bars->empty[s], 1);
      mbar_init(&bars->tail[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->accf[b], 1);
      mbar_init(&bars->acce[b], 8 * g.sets);   // the warps of both CTAs that write out
    }
    mbar_init(&bars->fin, 1);
    bars->abort = bars->stopped = 0;
    fence_mbar_init();
    prefetch_tmap(&mA);
    prefetch_tmap(&mB);
  }
  if (warp == 1) pair_tmem_alloc(&bars->tmem, 2 * kCols);
  tc_fence_before();
  cluster_sync_all();   // (the other CTA's shared memory is written from here on)
  tc_fence_after();
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 3) {
    // Each lane takes a run of experts.  (Rows out of the tensors, or before the
    // expert's first, are none of its.)
    const int per = (g.E + 31) / 32, e0 = min(lane * per, g.E), e1 = min(e0 + per, g.E);
    const int ft = feature_tiles(g);
    for (int e = e0; e < e1; ++e) {
      const long long b = min(max((long long)__ldg(g.off + e), 0ll), g.R);
      const long long n = max(min((long long)__ldg(g.off + e + 1), g.R) - b, 0ll);
      t.beg[e] = (int)b;
      t.cnt[e] = (int)n;
    }
    __syncwarp();
    // The widest tile: rounds of tiles at the cost of the widest, which below some
    // 160 rows is that of its features' loads.
    int cap = 256;
    if (g.what != 2) {
      long long best = 0x7FFFFFFFFFFFFFFFll;
      for (int c = 256; c >= 32; c -= 32) {
        int n = 0;
        for (int e = e0; e < e1; ++e) n += (t.cnt[e] + c - 1) / c;
        n = __reduce_add_sync(0xffffffffu, n);
        const long long cost = (n * (long long)ft + pairs - 1) / pairs * (max(c, 160) + 32);
        if (cost < best) {
          best = cost;
          cap = c;
        }
      }
    }
    int n = 0;
    for (int e = e0; e < e1; ++e) n += ((g.what == 2 ? g.N : t.cnt[e]) + cap - 1) / cap * ft;
    int s = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += v;
    }
    int at = s - n;
    for (int e = e0; e < e1; ++e) {
      t.pre[e] = at;
      at += ((g.what == 2 ? g.N : t.cnt[e]) + cap - 1) / cap * ft;
    }
    if (lane == 31) {
      t.pre[g.E] = s;
      bars->total = s;
      bars->cap = cap;
    }
    // A timeout recorded earlier stops this launch: one reading for both CTAs.
    if (lane == 0 && rank == 0 && g.status && *(volatile int*)g.status)
      for (int c = 0; c < 2; ++c) cluster_st(cluster_addr(&bars->stopped, c), 1);
  }
  cluster_sync_all();
  // (The same for all threads, as barriers of several warps follow: nothing writes `stopped` from
  // here on.  `abort` may be set by a wait of this launch before a thread comes to read it.)
  const uint32_t tmem = bars->tmem;
  const int cap = bars->cap, total = bars->stopped ? 0 : bars->total;

  if (warp == 0) {
    // ---------------- loads ----------------
    Ring rs;
    Walk walk(g);
    bool ok = true;
    for (int id = pair; id < total && ok; id += pairs) {
      const Tile q = walk.at(id, g, t, cap);
      const int half = q.nt / 2, beg = t.beg[q.e];
      const int fa = q.f0 + (int)rank * 128;
      const int nb = up32(half);   // rows of B, by boxes of 128, or of 64 and 32 (dW: features by boxes of 64)
      const uint32_t slice = kHalf + (g.what == 2 ? (uint32_t)(half + 63) / 64 * 8192u : (uint32_t)nb * 128u);
      for (int ks = 0; ks < q.steps; ++ks, rs.next(kStages)) {
        ok = wait_pair(&bars->empty[rs.slot], rs.phase ^ 1u, ab);
        if (!ok) break;
        if (g.stall) continue;
        if (lane == 0) {
          const bool clear = g.what == 2 && ks == q.steps - 1 && (q.last & 15) != 0;
          const int slices = ks == q.steps - 1 && q.last <= 64 ? 1 : 2;
          const uint32_t bar = clear ? cluster_addr(&bars->tail[rs.slot], rank) : cluster_addr(&bars->full[rs.slot], 0);
          cluster_arrive_expect_tx(bar, slices * slice);
          for (int sl = 0; sl < slices; ++sl) {
            unsigned char* a = smem + rs.slot * kStage + sl * kSlice;
            unsigned char* b = a + kHalf;
            const int k = ks * kStep + sl * 64;
            if (g.what == 0) {
              pair_load_3d(a, &mA, k, fa, q.e, bar);
            } else if (g.what == 1) {
              pair_load_3d(a, &mA, fa, k, q.e, bar);
              pair_load_3d(a + 8192, &mA, fa + 64, k, q.e, bar);
            } else {
              pair_load_2d(a, &mA, fa, beg + k, bar);
              pair_load_2d(a + 8192, &mA, fa + 64, beg + k, bar);
            }
            if (g.what == 2) {
              pair_load_2d(b, &mB, q.r0 + (int)rank * half, beg + k, bar);
              if (half > 64) pair_load_2d(b + 8192, &mB, q.r0 + (int)rank * half + 64, beg + k, bar);
            } else {
              const int y = beg + q.r0 + (int)rank * half;
              if (nb == 128) {
                pair_load_2d(b, &mB, k, y, bar);
              } else {
                if (nb >= 64) pair_load_2d(b, &mB64, k, y, bar);
                if (nb & 32) pair_load_2d(b + (nb & 64) * 128, &mB32, k, y + (nb & 64), bar);
              }
            }
          }
        }
        __syncwarp();
      }
    }
    // The arrivals under way at both CTAs' `empty` barriers land before either CTA ends.
    for (int i = 0; i < kStages && ok; ++i, rs.next(kStages)) ok = wait_pair(&bars->empty[rs.slot], rs.phase ^ 1u, ab);
  } else if (warp == 1 && rank == 0) {
    // ---------------- MMA issue, for both CTAs ----------------
    Ring rs, rb;
    Walk walk(g);
    bool ok = true;
    const uint32_t base = (1u << 4) | (DT == DETFFN_BF16 ? (1u << 7) | (1u << 10) : 0u) | (16u << 24) |
                          (g.what != 0 ? kIdescTransA : 0u) | (g.what == 2 ? kIdescTransB : 0u);
    const uint32_t astep = g.what != 0 ? 128u : 2u, bstep = g.what == 2 ? 128u : 2u;
    for (int id = pair; id < total && ok; id += pairs) {
      const Tile q = walk.at(id, g, t, cap);
      if (q.steps == 0) continue;
      ok = wait_pair(&bars->acce[rb.slot], rb.phase ^ 1u, ab);
      if (!ok) break;
      tc_fence_after();
      const uint32_t idesc = base | (uint32_t)(q.nt >> 3) << 17, acc = tmem + (uint32_t)(rb.slot * kCols);
      for (int ks = 0; ks < q.steps; ++ks, rs.next(kStages)) {
        ok = g.what == 2 && ks == q.steps - 1 ? wait_pair<true>(&bars->full[rs.slot], rs.phase, ab)
                                              : wait_pair(&bars->full[rs.slot], rs.phase, ab);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const int n = ks == q.steps - 1 ? (q.last + 15) / 16 : kStep / 16;
          for (int k0 = 0; k0 < n; k0 += 4) {
            unsigned char* a = smem + rs.slot * kStage + k0 / 4 * kSlice;
            const uint64_t da = g.what != 0 ? smem_desc_sw128_mn(a) : smem_desc_sw128(a);
            const uint64_t db = g.what == 2 ? smem_desc_sw128_mn(a + kHalf) : smem_desc_sw128(a + kHalf);
            for (int kk = 0; kk < 4 && k0 + kk < n; ++kk)
              pair_mma_f16(acc, da + (uint64_t)(astep * kk), db + (uint64_t)(bstep * kk), idesc, ks + k0 + kk > 0 ? 1u : 0u);
          }
          pair_commit(&bars->empty[rs.slot]);
          if (ks == q.steps - 1) pair_commit(&bars->accf[rb.slot]);
        }
        __syncwarp();
      }
      rb.next(2);
    }
    if (!ok) {   // stopped: the MMAs under way end before the shared memory is given up
      if (elect_one()) pair_commit(&bars->fin);
      __syncwarp();
      mbar_wait(&bars->fin, 0, kDefaultSpin, nullptr);
    }
  } else if (warp == 2 && g.what == 2) {
    // ---------------- rows beyond an expert's last, cleared ----------------
    Ring rs;
    Walk walk(g);
    uint32_t used = 0;   // parity of each stage's tail barrier
    for (int id = pair; id < total; id += pairs) {
      const Tile q = walk.at(id, g, t, cap);
      if (q.steps == 0 || (q.last & 15) == 0) {
        rs.adv(q.steps, kStages);
        continue;
      }
      rs.adv(q.steps - 1, kStages);
      if (!wait_pair(&bars->tail[rs.slot], used >> rs.slot & 1u, ab)) break;
      used ^= 1u << rs.slot;
      const int in = q.last % 64;   // rows of the last slice (not 0: a whole one needs no clearing)
      const int from = in * 128, to = (in + 15) / 16 * 2048, boxes = 2 + (q.nt / 2 + 63) / 64;
      unsigned char* a = smem + rs.slot * kStage + q.last / 64 * kSlice;
      for (int i = 0; i < boxes; ++i)
        for (int o = from + lane * 16; o < to; o += 512)
          *reinterpret_cast<uint4*>(a + i * 8192 + o) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) cluster_arrive(cluster_addr(&bars->full[rs.slot], 0));
      __syncwarp();
      rs.next(kStages);
    }
  } else if (warp >= 4) {
    // ---------------- outputs ----------------
    const int quarter = warp & 3, set = warp / 8;   // lanes of tensor memory; which chunks
    unsigned char* at = staged + set * kChunk * kPitch;
    Ring rb;
    Walk walk(g);
    for (int id = pair; id < total; id += pairs) {
      const Tile q = walk.at(id, g, t, cap);
      const int f = q.f0 + (int)rank * 128 + quarter * 32 + lane;
      uint16_t* out = g.out + (g.what == 2 ? q.e * g.stride + q.r0 * g.ldo : (t.beg[q.e] + (long long)q.r0) * g.ldo) + f;
      const bool in = f < g.F;
      if (q.steps == 0) {   // an empty sum
        const int x = lane % 16 * 8;
        if (!g.vec) {
          for (int i = 0; i < q.rows; ++i, out += g.ldo)
            if (in && set == 0) *out = 0;
        } else if (f - quarter * 32 - lane + x < g.F) {
          out += x - quarter * 32 - lane;
          for (int i = 2 * (warp - 4) + lane / 16; i < q.rows; i += 8 * g.sets)
            *reinterpret_cast<uint4*>(out + i * g.ldo) = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      // (One decision for the four warps: with barriers below, none may leave alone.)
      if (!out_all(set, wait_pair(&bars->accf[rb.slot], rb.phase, ab))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(rb.slot * kCols);
      out += set * kChunk * g.ldo;
      for (int c0 = set * kChunk; c0 < q.rows; c0 += g.sets * kChunk) {
        const int n = min(q.rows - c0, kChunk);
        if (g.vec) {
          // Through shared memory, [row][feature], by transposed matrix stores, and out
          // in vectors, two rows of 128 features to a store; element by element from
          // the registers a tile's 65536 results take 1024 stores of 64 bytes of each
          // CTA (dW of 16 experts of 94 rows, K = 1416, N = 4096: 92 and 59 us; 16384
          // rows of 16, K = 4096, N = 1536: 153 and 145 us).  A bulk copy for each row
          // takes some 100 cycles: 267 us of the first.
          uint32_t v[2][16];
          tmem_ld_frag(taddr + (uint32_t)c0, v[0]);
          tmem_ld_frag(taddr + (16u << 16) + (uint32_t)c0, v[1]);
          tmem_wait_ld();
          out_sync(set);   // (the last chunk's readers)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < 4; b += 2) {
              uint32_t w[4];
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const int i = 4 * (b + m / 2) + 2 * (m % 2);
                w[m] = Io<DT>::pair(__uint_as_float(v[h][i]), __uint_as_float(v[h][i + 1]));
              }
              const int row = 8 * (b + lane / 16) + lane % 8, feature = quarter * 32 + 16 * h + lane / 8 % 2 * 8;
              store_transposed(smem_u32(at + row * kPitch + feature * 2), w[0], w[1], w[2], w[3]);
            }
          out_sync(set);
          const int r = 8 * quarter + lane / 16, x = lane % 16 * 8;
          uint16_t* row = out - quarter * 32 - lane + x + r * g.ldo;
#pragma unroll
          for (int i = 0; i < 8; i += 2, row += 2 * g.ldo)
            if (r + i < n && f - quarter * 32 - lane + x < g.F)
              *reinterpret_cast<uint4*>(row) = *reinterpret_cast<const uint4*>(at + (r + i) * kPitch + x * 2);
        } else {
          uint32_t v[kChunk];
          tmem_ld32(taddr + (uint32_t)c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kChunk; ++i)
            if (i < n && in) Io<DT>::st(out + i * g.ldo, __uint_as_float(v[i]));
        }
        out += g.sets * kChunk * g.ldo;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) cluster_arrive_relaxed(cluster_addr(&bars->acce[rb.slot], 0));
      __syncwarp();
      rb.next(2);
    }
  }
  __syncwarp();
  // Stopped by a timeout: what copies are under way land (they take microseconds).
  if (*(volatile int*)ab.mine && total > 0 && !g.stall)
    for (int i = 0; i < 200; ++i) __nanosleep(10000);
  tc_fence_before();
  cluster_sync_all();   // (neither CTA's barriers or shared memory are used by the other from here on)
  tc_fence_after();
  if (warp == 1) pair_tmem_dealloc(tmem, 2 * kCols);
}

int smem_bytes(int E) { return 1024 + kStages * kStage + kOutBytes + (int)((sizeof(Bars) + 127) & ~127) + tables_bytes(E); }

template <int DT>
cudaError_t run(const GroupedArgs& a, Grouped what, const Waits& wt, int sm_count, cudaStream_t st) {
  static PerDevice ready;
  const cudaError_t e = once_per_device(ready, [] {
    return cudaFuncSetAttribute(k_grouped_tc<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kGroupedMaxExperts));
  });
  if (e != cudaSuccess) return e;
  const bool f16 = DT == DETFFN_F16;
  // (The stride of a single row is never used; the tensor map wants a multiple of 16 bytes.)
  const long long ldx = a.R > 1 ? a.x.ld : grouped_pad(a.K), ldd = a.R > 1 ? a.dout.ld : grouped_pad(a.N);
  const long long ldw = a.E * a.N > 1 ? a.ldw : grouped_pad(a.K);
  const long long dw[3] = {a.K, a.N, a.E}, sw[2] = {ldw, a.N * ldw};
  CUtensorMap mA, mB, mB64, mB32;
  Args g{};
  bool ok;
  long long rt;
  auto rows_maps = [&](const void* p, long long width, long long ld) {
    return tc_make_map_rows(&mB, f16, p, a.R, width, ld, 64, 128) && tc_make_map_rows(&mB64, f16, p, a.R, width, ld, 64, 64) &&
           tc_make_map_rows(&mB32, f16, p, a.R, width, ld, 64, 32);
  };
  if (what == Grouped::kForward) {
    const int box[3] = {64, 128, 1};
    ok = tc_make_map_3d(&mA, f16, a.W, dw, sw, box) && rows_maps(a.x.p, a.K, ldx);
    g.what = 0, g.F = (int)a.N, g.C = (int)a.K, g.out = static_cast<uint16_t*>(const_cast<void*>(a.out.p)), g.ldo = a.out.ld;
    rt = a.R / 32 + a.E;
  } else if (what == Grouped::kInput) {
    const int box[3] = {64, 64, 1};
    ok = tc_make_map_3d(&mA, f16, a.W, dw, sw, box) && rows_maps(a.dout.p, a.N, ldd);
    g.what = 1, g.F = (int)a.K, g.C = (int)a.N, g.out = static_cast<uint16_t*>(const_cast<void*>(a.dx.p)), g.ldo = a.dx.ld;
    rt = a.R / 32 + a.E;
  } else {
    ok = tc_make_map_rows(&mA, f16, a.x.p, a.R, a.K, ldx, 64, 64) && tc_make_map_rows(&mB, f16, a.dout.p, a.R, a.N, ldd, 64, 64);
    mB64 = mB32 = mB;
    g.what = 2, g.F = (int)a.K, g.N = (int)a.N, g.out = static_cast<uint16_t*>(a.dW), g.ldo = a.K, g.stride = a.N * a.K;
    rt = (a.N + 255) / 256 * a.E;
  }
  if (!ok) return cudaErrorInvalidValue;
  // Contractions of up to 4 stages on average: the results' way out bounds them
  // (kMostThreads: dW of 16 experts of 94 rows, K = 1416, N = 4096: 79 and 69 us); with
  // long ones four more warps cost 2 % (16384 rows, K = 4096, N = 1536).
  g.sets = (what == Grouped::kWeight ? a.R / a.E : (long long)g.C) <= 256 ? 2 : 1;
  const bool one = what != Grouped::kWeight && a.R == 1;
  g.vec = (uintptr_t)g.out % 16 == 0 && g.F % 8 == 0 && (one || g.ldo % 8 == 0);
  g.E = a.E;
  g.R = a.R;
  g.off = a.off;
  g.status = wt.status;
  g.spin = wt.spin;
  g.stall = wt.stall;
  const long long most = rt * ((g.F + 255) / 256), slots = sm_count / 2;
  const int pairs = (int)(most < slots ? most : slots);
  return launch_cluster(k_grouped_tc<DT>, dim3(2 * pairs), g.sets == 2 ? kMostThreads : kThreads, smem_bytes(a.E), 2, st, mA, mB,
                        mB64, mB32, g);
}

}  // namespace

cudaError_t launch_grouped_tensor(const GroupedArgs& a, Grouped what, const Waits& wt, int sm_count, cudaStream_t st) {
  return a.dtype == DETFFN_F16 ? run<DETFFN_F16>(a, what, wt, sm_count, st) : run<DETFFN_BF16>(a, what, wt, sm_count, st);
}

}  // namespace detffn
