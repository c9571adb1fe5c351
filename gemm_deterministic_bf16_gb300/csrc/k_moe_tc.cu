// k_moe_tc.cu -- the mixture-of-experts layer for a few tokens on the tensor
// cores, BF16 and FP16 (the formulas are those of k_moe.cu).
//
// One persistent launch, one CTA per SM, after the router's logits.  Every
// CTA works the routing out for itself from the logits (one warp per token),
// so that nothing is handed over through memory, then takes units in turn:
//   gate/up: 64 rows of Wg[e] over the same 64 rows of Wu[e] (the MMA's 128
//     rows) times the expert's tokens, K = H; h for those 64 features.  Where
//     that makes few units, 32 rows of each and twice the K to a stage: the
//     MMA's other rows then read what follows and are not used
//   down:    128 rows of Wd[e] times the expert's rows of h, K = I or a part of
//     it; partial outputs y of the pairs
// All gate/up units come before all down units, experts in ascending order.
// A down unit waits (bounded) until its expert's gate/up units are counted,
// with its first weight tiles already on their way.  Those units were claimed
// earlier, by CTAs that are running and wait for nothing themselves, so the
// wait ends whatever else holds the other SMs.  At the end all CTAs add the
// pairs of each token, in the order of its choices, as the 128-feature tiles of
// the output are counted complete (left to the CTA that counts a tile last,
// that alone took 18 us for 64 tokens of 64 experts).
//
// The down projection's K is cut where H gives few tiles (into as many parts
// as make 16 units of an expert, of two stages or more): one CTA alone is slow
// to stream a whole row tile, as its ring holds six stages.  Four tokens of 6
// experts, H = 616, I = 1376: 20.2 us whole, 16.1 in parts.  The cut depends
// on H and I alone, and the parts are added in order.
//
// The work is the weights' bytes: each active expert's are read once, by TMA
// boxes of 64 K (128-byte swizzle) into a ring of stages of 32 KB of weights.
// A gate/up unit multiplies them with the rows of all tokens, one box a slice,
// and leaves the columns of other experts' tokens aside: a row gather of the
// expert's own tokens holds the TMA unit for some 40 ns per four rows (64
// tokens of 2 experts, H = 4096, I = 1024: 75 us gathered, 39 so; 55 of 11
// experts: 74 and 59; 64 of 64 experts, 6 choices, 6.5 tokens an expert on
// average: 371 and 369), and the MMA's time does not depend on its columns up
// to 32.  A down unit's pairs are neighbours in h, and one box of 8, 16, 32 or
// 64 rows takes them; the rows past the unit's are other units' and are not
// used, whatever they hold.  h goes to the down projection as two terms, its
// rounding to the stored type and the rounding of what that left, in columns of
// their own, which meet when y is read out: with one term the rounding of h
// alone doubles the variance of out's error (1.41 times the error of one
// rounding, measured), and the second costs only tensor time, which is idle
// here.  BF16 has FP32's range, so the two hold 16 bits of any h.  FP16 has
// not: each term has a power of two of its own (Terms below), which holds 16
// bits of h from 2^-13 to 2^23 and 2^-29 below.  A pair whose largest |h| lies
// outside that range (or is not finite) is multiplied again at the end, on the
// CUDA cores from h in FP32; its columns on the tensor cores are not used (one
// token, 8 of 128 experts, H = 2048, I = 768: 28 us, and 313 with all pairs again;
// 64 tokens, 6 of 64, H = 4096, I = 1536: 370 and 2041).  A
// row's sum over K is one accumulation in FP32 in tensor memory, whatever the
// other columns are, so a token's result does not depend on the other tokens.
//
// HBM bounds it once the weights take longer than the chain around them (of the
// measured copy rate: 64 tokens, 6 of 64 experts, H = 4096, I = 1536, 2.4 GB of
// weights: 367 us, 98 %; 7 tokens, 2 of 16, I = 1416: 59 to 66 us by the
// experts hit, 75 to 85 %).  Below that the chain does: one token, 8 of 128, H =
// 2048, I = 768 takes 27.2 us, 11.4 of them for the weights; 1.5 us for the
// logits, 3 for the routing, 2 to 3 until the first stage, 8 of gate/up, 3 until
// h is seen, 3 of down, 4 for the sums.
#include "elt.cuh"
#include "moe.cuh"
#include "ptx.cuh"
#include "tc.h"

namespace detffn {
namespace {

// Instruction descriptor, kind::f16: FP32 accumulator, BF16 or FP16 operands,
// both K-major, M x N tile.
__device__ constexpr uint32_t idesc_f16(bool bf16, int M, int N) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

static_assert(kMoeMaxTokens <= 64, "16 warps take four tokens each; an expert's tokens are 64 bits");
constexpr int kThreads = 512;     // all work out the routing; then warp 0 loads, warp 1 issues MMAs, warps
                                  // 4-7 read the sums, 8-15 form the routing weights, and 4-15 out
constexpr int kEpi0 = 4;          // first epilogue warp (its TMEM lane quarter is warp % 4)
constexpr int kHelpers = kThreads / 32 - kEpi0 - 4;  // warps that form the routing weights
constexpr int KS = 128;           // K positions of a down unit's stage
constexpr int kBoxBytes = 64 * 128;              // 64 rows x 64 K
constexpr int kWeightBytes = 4 * kBoxBytes;      // 128 rows x 128 K
constexpr int kMaxStages = 8;
constexpr int kSmemMax = 227 * 1024;
constexpr int kUnits = 4;                        // units a CTA has claimed and not finished, at most
constexpr int kXch = 128 * 8 * 4;                // gate and up values of eight tokens

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], accf[2], acce[2], ufull[kUnits], uempty[kUnits], weights, done, fin;
  uint32_t tmem;
  int abort, go;
  int unit[kUnits];  // claimed units; past the last: no more
  int active;   // experts with tokens
  int most;     // most tokens of one expert
};

struct Args {
  MoeArgs m;
  int cols;          // most columns of a unit's sums
  int ring;          // bytes for stages
  int tb;            // down tiles of an expert
  int parts, kpart;  // parts of a down tile's K, stages of a part
  int* claim;        // units claimed by all CTAs
  int* ready;        // [E] gate/up units done
  int* tickets;      // [tb] down units done
  float* y;          // [parts][T * k][H]
  unsigned* top;     // [T * k] FP16: bits of the largest |h| of each pair
  float* h32;        // [T * k][I] FP16: h
  int* status;
  long long spin;
  int stall;
};

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, long long limit, volatile int* abort_flag,
                                              int* status) {
  for (long long i = 0; i < limit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023) == 1023 && *abort_flag) return false;
  }
  *abort_flag = 1;
  if (status) atomicExch(status, (int)DETFFN_ERR_TIMEOUT);
  return false;
}

__device__ __forceinline__ void tma_load_3d_hint(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
      "%4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same barrier; whether `ok` held in all 128 threads.
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// The routing tables in shared memory.  A token takes an expert once, so an
// expert's tokens are a mask of 64 bits, and a pair's place among the pairs
// ordered by expert and token is the expert's first plus a count of bits.
struct Tables {
  unsigned long long* mask;   // [E] tokens of each expert
  int* first;       // [E + 1] first pair of each expert
  int* act;         // [E] active experts, ascending
  float* l;         // [P] chosen logits by pair (token * k + slot)
  float* w;         // [P] weights by pair
  uint16_t* id;     // [P] expert by pair
  uint16_t* pos;    // [P] place of a pair
};
__host__ __device__ inline int tables_bytes(int E, int P) {
  return ((4 * E + 1 + 2 * P) * 4 + 2 * P * 2 + 15) & ~15;
}
__device__ __forceinline__ Tables tables_at(unsigned char* p, int E, int P) {
  Tables t;
  t.mask = reinterpret_cast<unsigned long long*>(p);
  t.first = reinterpret_cast<int*>(t.mask + E);
  t.act = t.first + E + 1;
  t.l = reinterpret_cast<float*>(t.act + E);
  t.w = t.l + P;
  t.id = reinterpret_cast<uint16_t*>(t.w + P);
  t.pos = t.id + P;
  return t;
}

// h as two terms of the stored type, and y of the two terms' sums.
template <int DT> struct Terms;
template <> struct Terms<DETFFN_BF16> {
  static constexpr float kMax = 0x1.fep127f;   // the largest BF16: h may round beyond it
  __device__ static float first(float h) { return Io<DETFFN_BF16>::round(fminf(fmaxf(h, -kMax), kMax)); }
  // (An infinity or a NaN of h is the second term's.)
  __device__ static float second(float h, float first) { return h - first; }
  __device__ static float sum(float y1, float y2) { return y1 + y2; }
};
template <> struct Terms<DETFFN_F16> {
  // Of |h| <= 2^23 the first is at most 2^15, and the second, 16 times what its
  // rounding left (half of 2^4 2^8 at most), too.
  static constexpr float kTop = 0x1p23f, kLow = 0x1p-13f;   // the largest |h| of a pair that they are for
  __device__ static float first(float h) { return Io<DETFFN_F16>::round(h * 0x1p-8f); }
  __device__ static float second(float h, float first) { return (h - first * 0x1p8f) * 0x1p4f; }
  __device__ static float sum(float y1, float y2) { return fmaf(y1, 0x1p8f, y2 * 0x1p-4f); }
  // `top`: bits of a pair's largest |h|.
  __device__ static bool hold(uint32_t top) {
    return top == 0u || (top >= __float_as_uint(kLow) && top <= __float_as_uint(kTop));
  }
};

// y of one pair on the CUDA cores: products of h in FP32 with `rows` (at most
// 128) rows of weights, by one warp; lane l ends with those of rows 4 l ..
// 4 l + 3.  Out of line, as it is hardly ever called.
template <int DT>
__device__ __noinline__ float4 down_rows(const typename Io<DT>::E* w, const float* h, long long I, int rows, int lane) {
  float4 mine = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int f = 0; 4 * f < rows; ++f, w += 4 * I) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (long long k = 8 * lane; k < I; k += 256) {
      const float4 a0 = __ldcg(reinterpret_cast<const float4*>(h + k)), a1 = __ldcg(reinterpret_cast<const float4*>(h + k) + 1);
      const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float b[8];
        Io<DT>::ld8(w + i * I + k, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i] = fmaf(a[j], b[j], s[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = warp_sum(s[i]);
    if (lane == f) mine = make_float4(s[0], s[1], s[2], s[3]);
  }
  return mine;
}

// Rows of h that a down unit of n pairs loads, by one box.
__host__ __device__ inline int hrows(int n) { return n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64; }

struct Unit {
  bool down;
  int a, tile, part, e, p0, n;   // active index, tile of the expert, part of K, expert, first pair, pairs
};
__device__ __forceinline__ Unit unit_at(int u, const Args& g, const Tables& t, int active, int ta) {
  Unit r;
  const int na = active * ta;
  r.down = u >= na;
  const int v = r.down ? u - na : u;
  const int per = r.down ? g.tb * g.parts : ta;
  r.a = v / per;
  r.tile = v - r.a * per;
  r.part = 0;
  if (r.down) {
    r.part = r.tile / g.tb;
    r.tile -= r.part * g.tb;
  }
  r.e = t.act[r.a];
  r.p0 = t.first[r.e];
  r.n = t.first[r.e + 1] - r.p0;
  return r;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
    k_moe(const __grid_constant__ CUtensorMap mWg, const __grid_constant__ CUtensorMap mWu,
          const __grid_constant__ CUtensorMap mWg32, const __grid_constant__ CUtensorMap mWu32,
          const __grid_constant__ CUtensorMap mWd, const __grid_constant__ CUtensorMap mX,
          const __grid_constant__ CUtensorMap mH8, const __grid_constant__ CUtensorMap mH16,
          const __grid_constant__ CUtensorMap mH32, const __grid_constant__ CUtensorMap mH64,
          const __grid_constant__ Args g) {
  using El = typename Io<DT>::E;
  extern __shared__ unsigned char raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  const MoeArgs& m = g.m;
  const int P = m.T * m.k;
  Bars* bars = reinterpret_cast<Bars*>(smem + g.ring);
  float* xch = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(bars) + ((sizeof(Bars) + 127) & ~127));
  const Tables t = tables_at(reinterpret_cast<unsigned char*>(xch) + kXch, m.E, P);
  volatile int* abort_flag = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = g.spin > 0 ? g.spin : kDefaultSpin;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->accf[b], 1);
      mbar_init(&bars->acce[b], 4);
    }
    for (int q = 0; q < kUnits; ++q) {
      mbar_init(&bars->ufull[q], 1);
      mbar_init(&bars->uempty[q], 5);   // the MMA warp and four epilogue warps
    }
    mbar_init(&bars->weights, kHelpers);
    mbar_init(&bars->done, 1);
    mbar_init(&bars->fin, 1);
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&mWg);
    prefetch_tmap(&mWu);
    prefetch_tmap(&mWd);
    prefetch_tmap(&mX);
    prefetch_tmap(&mH8);
  }
  const uint32_t tcols = g.cols <= 16 ? 32 : g.cols <= 32 ? 64 : g.cols <= 64 ? 128 : 256;  // two units' sums
  if (warp == 1) {
    tmem_alloc(&bars->tmem, tcols);
    tmem_relinquish();
  }
  for (int e = threadIdx.x; e < m.E; e += kThreads) t.mask[e] = 0;
  grid_dep_wait();
  grid_dep_launch();

  // The first claim, and whether a timeout recorded earlier stops this launch:
  // under way during the routing.
  int claimed = 0, stopped = 0;
  if (threadIdx.x == 0) {
    claimed = atomicAdd(g.claim, 1);
    if (g.status) stopped = *(volatile int*)g.status;
  }

  // ---------------- the routing ----------------
  const int ld = (m.E + 3) & ~3;   // (past the last expert: 0, below every key)
  const int items = (m.T * ld + kThreads - 1) / kThreads;
  if (items * ld <= 24 * m.k + 40) {
    // Every logit's rank by comparing it with its token's, a thread to a logit:
    // about 10 instructions a pair of logits for each of a thread's items, where
    // the rounds below take 240 a choice.  From the logits to the counts, 2 us of
    // other work included: 55 tokens of 11 experts, 5 choices, 3.3 us, and by
    // rounds 6.1; 49 of 38 experts 6.2 by ranks, and 64 of 64, 6 choices, 6.5 by
    // rounds.
    uint32_t* key = reinterpret_cast<uint32_t*>(smem);   // (the stages' memory)
#pragma unroll 4
    for (int i = threadIdx.x; i < m.T * ld; i += kThreads) {
      const int q = i / ld, e = i - q * ld;
      key[i] = e < m.E ? moe_key(__ldcg(m.logits + (long long)q * m.E + e)) : 0u;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m.T * ld; i += kThreads) {
      const int q = i / ld, e = i - q * ld;
      const uint32_t mine = key[i];
      if (mine == 0u) continue;
      int rank = 0;
      for (int f = 0; f < ld; f += 4) {
        // A larger key comes first, and an equal one of a lower expert.
        const uint4 o = *reinterpret_cast<const uint4*>(key + q * ld + f);
        rank += (o.x + (f < e ? 1u : 0u) > mine) + (o.y + (f + 1 < e ? 1u : 0u) > mine) +
                (o.z + (f + 2 < e ? 1u : 0u) > mine) + (o.w + (f + 3 < e ? 1u : 0u) > mine);
      }
      if (rank < m.k) {
        t.id[q * m.k + rank] = (uint16_t)e;
        t.l[q * m.k + rank] = moe_logit(mine);
      }
    }
  } else if (m.E <= 128) {
    // Rounds, up to four tokens of a warp side by side.
    constexpr int kWarps = kThreads / 32;
    uint32_t key[4][4];
    MoeChoice c[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) moe_keys<4>(m.logits, m.T, m.E, warp + b * kWarps, lane, key[b]);
    moe_choose<4, 4>(key, m.k, lane, c);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int q = warp + b * kWarps;
      if (q < m.T && lane < m.k) {
        t.id[q * m.k + lane] = (uint16_t)c[b].expert;
        t.l[q * m.k + lane] = c[b].logit;
      }
    }
  } else {
    for (int q = warp; q < m.T; q += kThreads / 32) {
      uint32_t key[1][kMoeMaxExperts / 32];
      MoeChoice c[1];
      moe_keys<kMoeMaxExperts / 32>(m.logits, m.T, m.E, q, lane, key[0]);
      moe_choose<kMoeMaxExperts / 32, 1>(key, m.k, lane, c);
      if (lane < m.k) {
        t.id[q * m.k + lane] = (uint16_t)c[0].expert;
        t.l[q * m.k + lane] = c[0].logit;
      }
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += kThreads) {
    const int q = p / m.k, e = t.id[p];
    atomicOr(&t.mask[e], 1ull << q);
  }
  __syncthreads();
  if (warp == 0) {
    // Exclusive sums of the counts and the list of active experts: a lane
    // takes a run of experts.
    const int per = (m.E + 31) / 32, e0 = lane * per, e1 = min(m.E, e0 + per);
    int c = 0, on = 0, most = 0;
#pragma unroll 4
    for (int e = e0; e < e1; ++e) {
      const int n = __popcll(t.mask[e]);
      c += n;
      on += n > 0;
      most = max(most, n);
    }
    int s = c | on << 16;   // (at most 1024 pairs, 512 experts)
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += v;
    }
    int at = (s & 0xFFFF) - c, na = (s >> 16) - on;
    for (int e = e0; e < e1; ++e) {
      const int n = __popcll(t.mask[e]);
      t.first[e] = at;
      at += n;
      if (n > 0) t.act[na++] = e;
    }
    most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
    if (lane == 31) {
      t.first[m.E] = at;
      bars->active = na;
      bars->most = most;
    }
  }
  fence_proxy_async_smem();  // (the stages' memory held keys until here)
  tc_fence_before();
  if (threadIdx.x == 0) bars->go = stopped == 0;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const int active = bars->active;
  // Rows of Wg and of Wu in a gate/up unit, and the units of an expert.  An MMA
  // costs about 75 cycles whatever its columns (up to 32), so half-filled ones
  // halve what a CTA can take in, and pay where units of 64 rows fill the grid
  // badly: at most half of it (one token of 2 experts, H = 4096, I = 1024: 27.7
  // us with 64 rows, 25.3 with 32), or once and at most half of it again, with
  // rows long enough (7 tokens of 16 experts, H = 4096, I = 1416: 62.3 and 59.4;
  // 32 of 8, 4 choices, H = 7168, I = 1248: 95 and 86; H = 1024: even).
  // Elsewhere they cost 2 to 16 % (54 of 78, 663 units: 43.9 and 51.1).
  const int wide = active * (int)((m.I + 63) / 64), grid = (int)gridDim.x;
  const bool few = 2 * wide <= grid || (wide > grid && 2 * wide <= 3 * grid && m.H >= 2048);
  const int R = few ? 32 : 64, ta = (int)((m.I + R - 1) / R);
  // A stage: 32 KB of weights as slices of 64 K, then a token tile for each
  // slice: of x (all tokens, in whole sixteens), or the first terms of h and
  // then the second, as this call's largest expert needs them.  With up to 16
  // tokens, eight of an expert, six stages fit.
  const int SL = 128 / R;   // slices of a gate/up stage; a down unit's has two
  const int xtile = (m.T + 15) / 16 * 2048, htile = 256 * hrows(bars->most);
  const int stage_bytes = kWeightBytes + max(SL * xtile, 2 * htile);
  const int NS = min(kMaxStages, g.ring / stage_bytes);
  const int units = bars->go ? active * (ta + g.tb * g.parts) : 0;
  const int ka = (int)((m.H + 64 * SL - 1) / (64 * SL)), kb = (int)((m.I + KS - 1) / KS);

  if (warp == 0) {
    // ---------------- loads ----------------
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    Ring rs, ru;
    long long issued = 0;  // stages whose weights went out
    bool ok = true;
    auto stage = [&](int s) { return smem + (size_t)s * stage_bytes; };
    int u = __shfl_sync(0xffffffffu, claimed, 0);
    while (true) {
      // Hand the claimed unit (or the end) to the other warps.
      if (!__all_sync(0xffffffffu, wait_or_abort(&bars->uempty[ru.slot], ru.phase ^ 1u, limit, abort_flag, g.status))) break;
      if (lane == 0) {
        bars->unit[ru.slot] = u;
        mbar_arrive(&bars->ufull[ru.slot]);
      }
      __syncwarp();
      ru.next(kUnits);
      if (u >= units) break;
      const Unit q = unit_at(u, g, t, active, ta);
      const int k0 = q.part * g.kpart, nk = q.down ? min(g.kpart, kb - k0) : ka, rows = hrows(q.n);
      const uint32_t bytes = (uint32_t)kWeightBytes + (uint32_t)(q.down ? 512 * rows : SL * xtile);
      auto weights = [&](int ks, Ring r) -> bool {
        const bool wok = wait_or_abort(&bars->empty[r.slot], r.phase ^ 1u, limit, abort_flag, g.status);
        if (!__all_sync(0xffffffffu, wok)) return false;
        if (g.stall) return true;
        unsigned char* d = stage(r.slot);
        uint64_t* bar = &bars->full[r.slot];
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, bytes);
          if (q.down) {
            for (int i = 0; i < 4; ++i)  // box i: K half i / 2, rows 64 (i % 2)
              tma_load_3d_hint(d + i * kBoxBytes, &mWd, (k0 + ks) * KS + (i >> 1) * 64, q.tile * 128 + (i & 1) * 64, q.e, bar, pol);
          } else if (R == 64) {
            for (int i = 0; i < 2; ++i) {
              tma_load_3d_hint(d + 2 * i * kBoxBytes, &mWg, ks * KS + i * 64, q.tile * 64, q.e, bar, pol);
              tma_load_3d_hint(d + (2 * i + 1) * kBoxBytes, &mWu, ks * KS + i * 64, q.tile * 64, q.e, bar, pol);
            }
          }
        }
        __syncwarp();
        if (!q.down && R < 64 && lane < 8) {
          // Boxes of 32 rows, one a lane: slice, weight.
          const int sl = lane >> 1, up = lane & 1;
          tma_load_3d_hint(d + sl * R * 256 + up * R * 128, up ? &mWu32 : &mWg32, (ks * SL + sl) * 64, q.tile * R, q.e, bar, pol);
        }
        __syncwarp();
        return true;
      };
      auto tokens = [&](int ks, Ring r) {
        if (g.stall) return;
        unsigned char* d = stage(r.slot) + kWeightBytes;
        uint64_t* bar = &bars->full[r.slot];
        if (q.down) {
          // K half, term: the second terms' rows follow the first terms' of this unit.
          if (lane < 4)
            tma_load_2d(d + (lane & 1) * htile + (lane >> 1) * rows * 128,
                        rows == 8 ? &mH8 : rows == 16 ? &mH16 : rows == 32 ? &mH32 : &mH64,
                        (k0 + ks) * KS + (lane & 1) * 64, (lane >> 1) * P + q.p0, bar);
        } else if (lane < SL) {
          tma_load_2d(d + lane * xtile, &mX, (ks * SL + lane) * 64, 0, bar);
        }
        __syncwarp();
      };
      // A down unit's first weight tiles go out before the wait for h.
      int ahead = 0;
      Ring w = rs;
      if (q.down) {
        for (; ahead < nk && ahead < NS && ok; ++ahead, w.next(NS)) {
          ok = weights(ahead, w);
          if (!ok) break;
          ++issued;
        }
        bool rok = ok;
        if (ok && lane == 0) {
          long long i = 0;
          for (; i < limit; ++i) {
            if (ld_acquire(g.ready + q.e) >= ta) break;
            if ((i & 255) == 255 && *abort_flag) {
              i = limit;
              break;
            }
            __nanosleep(32);
          }
          if (i >= limit) {
            rok = false;
            *abort_flag = 1;
            if (g.status) atomicExch(g.status, (int)DETFFN_ERR_TIMEOUT);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)rok, 0) != 0;
        __syncwarp();                // (lane 0's acquire comes before the loads of all; a shuffle orders no memory)
        fence_proxy_async_global();  // the TMA loads below read what generic stores wrote
        if (ahead == nk && lane == 0) claimed = atomicAdd(g.claim, 1);
        // (Also after a stop: stages with their weights out get their tokens, so that each completes.)
        for (int ks = 0; ks < ahead; ++ks, rs.next(NS)) tokens(ks, rs);
      }
      for (int ks = ahead; ks < nk && ok; ++ks, rs.next(NS)) {
        // The next unit is claimed with this one's last loads: earlier, a CTA
        // that waits for h would hold a second unit that an idle one could take.
        if (ks == nk - 1 && lane == 0) claimed = atomicAdd(g.claim, 1);
        ok = weights(ks, rs);
        if (!ok) break;
        ++issued;
        tokens(ks, rs);
      }
      if (!ok) break;
      u = __shfl_sync(0xffffffffu, claimed, 0);
    }
    // Drain: every stage that was filled has landed (long bound).
    if (!g.stall && lane == 0) {
      Ring r;
      for (long long i = 0; i < issued; ++i, r.next(NS))
        if (i + NS >= issued) mbar_wait(&bars->full[r.slot], r.phase, kDefaultSpin, nullptr);
    }
  } else if (warp == 1) {
    // ---------------- MMA issue ----------------
    Ring rs, rb, ru;
    bool ok = true;
    while (true) {
      bool wok = wait_or_abort(&bars->ufull[ru.slot], ru.phase, limit, abort_flag, g.status);
      if (!__all_sync(0xffffffffu, wok)) break;
      const int u = bars->unit[ru.slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->uempty[ru.slot]);
      ru.next(kUnits);
      if (u >= units) break;
      const Unit q = unit_at(u, g, t, active, ta);
      const int nk = q.down ? min(g.kpart, kb - q.part * g.kpart) : ka;
      const uint32_t idesc = idesc_f16(DT == DETFFN_BF16, 128, q.down ? 2 * hrows(q.n) : (m.T + 15) / 16 * 16);
      const uint32_t acc = tmem + (uint32_t)(rb.slot * g.cols);
      wok = wait_or_abort(&bars->acce[rb.slot], rb.phase ^ 1u, limit, abort_flag, g.status);
      ok = __all_sync(0xffffffffu, wok) != 0;
      for (int ks = 0; ks < nk && ok; ++ks, rs.next(NS)) {
        wok = wait_or_abort(&bars->full[rs.slot], rs.phase, limit, abort_flag, g.status);
        if (!__all_sync(0xffffffffu, wok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        unsigned char* d = smem + (size_t)rs.slot * stage_bytes;
        if (elect_one()) {
          const int slices = q.down ? 2 : SL, wstep = q.down ? 128 * 128 : R * 256, tstep = q.down ? htile : xtile;
          for (int sl = 0; sl < slices; ++sl) {
            const uint64_t da = smem_desc_sw128(d + sl * wstep);
            const uint64_t db = smem_desc_sw128(d + kWeightBytes + sl * tstep);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_bf16(acc, da + 2u * kk, db + 2u * kk, idesc, ks > 0 || sl > 0 || kk > 0 ? 1u : 0u);
          }
          tc_commit(&bars->empty[rs.slot]);
          if (ks == nk - 1) tc_commit(&bars->accf[rb.slot]);
        }
        __syncwarp();
      }
      if (!ok) break;
      rb.next(2);
    }
    if (elect_one()) tc_commit(&bars->fin);
    __syncwarp();
    if (lane == 0) mbar_wait(&bars->fin, 0, kDefaultSpin, nullptr);
  } else if (warp >= kEpi0 + 4) {
    // ---------------- weights and places of the pairs, wanted only at the end ----------------
    for (int q = warp - kEpi0 - 4; q < m.T; q += kHelpers) {
      const float all = m.normalize ? -1.0f : moe_sum(m.logits + (long long)q * m.E, m.E, t.l[q * m.k], lane);
      const int p = q * m.k + lane;
      if (lane < m.k) {
        const float w = moe_weight(t.l + q * m.k, m.k, lane, all);
        const int e = t.id[p];
        t.w[p] = w;
        t.pos[p] = (uint16_t)(t.first[e] + __popcll(t.mask[e] & ((1ull << q) - 1ull)));
        if (blockIdx.x == 0) {
          m.experts[p] = e;
          m.weights[p] = w;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->weights);
  } else if (warp >= kEpi0 && warp < kEpi0 + 4) {
    // ---------------- outputs ----------------
    const int quarter = warp & 3, row = quarter * 32 + lane, et = threadIdx.x - kEpi0 * 32;
    Ring rb, ru;
    for (;; rb.next(2)) {
      // The next unit, and its sums.
      bool aok = wait_or_abort(&bars->ufull[ru.slot], ru.phase, limit, abort_flag, g.status);
      const int u = aok ? bars->unit[ru.slot] : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->uempty[ru.slot]);
      ru.next(kUnits);
      const Unit q = unit_at(aok && u < units ? u : 0, g, t, active, ta);
      if (aok && u < units) aok = wait_or_abort(&bars->accf[rb.slot], rb.phase, limit, abort_flag, g.status);
      // One decision for the four warps: with a barrier each below, none may
      // leave alone.
      if (!epi_all(aok) || u >= units) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(rb.slot * g.cols);
      // The columns that hold pairs of this expert.
      const unsigned long long cols = q.down ? ~0ull >> (64 - q.n) : t.mask[q.e];
      for (int c0 = 0; c0 < 64 && cols >> c0; c0 += 8) {
        const unsigned here = (unsigned)(cols >> c0) & 0xFFu;
        if (here == 0u) continue;
        uint32_t v[8];
        tmem_ld8(taddr + (uint32_t)c0, v);
        if (q.down) {
          uint32_t v2[8];   // the second terms' part
          tmem_ld8(taddr + (uint32_t)(hrows(q.n) + c0), v2);
          tmem_wait_ld();
          const long long r = q.tile * 128ll + row;
          if (r < m.H) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (here >> i & 1)
                g.y[((long long)q.part * P + q.p0 + c0 + i) * m.H + r] =
                    Terms<DT>::sum(__uint_as_float(v[i]), __uint_as_float(v2[i]));
          }
        } else {
          // Gate rows are lanes 0 .. R - 1 of tensor memory and up rows R .. 2 R -
          // 1: they meet in shared memory, and all threads take (feature, token)
          // pairs.
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) xch[i * 128 + row] = __uint_as_float(v[i]);
          epi_sync();
          const int f = et & (R - 1);
          const long long r = q.tile * (long long)R + f;
          const bool in = r < m.I;
#pragma unroll 1
          for (int i0 = et / R; i0 < 8; i0 += 256 / R) {
            float gt[2], hv[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float* at = xch + (i0 + b * (128 / R)) * 128 + f;
              gt[b] = at[0];
              hv[b] = at[R];
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) hv[b] *= gt[b] * sigma<false>(gt[b]).s;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int i = i0 + b * (128 / R);   // (the same in all threads of a warp)
              if (!(here >> i & 1)) continue;
              const int place = q.p0 + __popcll(cols & ((1ull << (c0 + i)) - 1ull));
              if constexpr (DT == DETFFN_F16) {
                const unsigned top = __reduce_max_sync(0xffffffffu, in ? __float_as_uint(fabsf(hv[b])) : 0u);
                if (lane == 0) atomicMax(g.top + place, top);
                if (in) g.h32[place * m.I + r] = hv[b];
              }
              if (in) {
                El* at = static_cast<El*>(m.h) + place * m.I + r;
                const float first = Terms<DT>::first(hv[b]);
                Io<DT>::st(at, first);
                Io<DT>::st(at + P * m.I, Terms<DT>::second(hv[b], first));
              }
            }
          }
          epi_sync();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->acce[rb.slot]);
      if (q.down) {
        // This unit's part of y is written: count it.
        epi_sync();
        if (et == 0) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(g.tickets + q.tile) : "memory");
      } else {
        // h of this tile is written: count it.
        fence_proxy_async_global();
        epi_sync();
        if (et == 0) {
          asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(g.ready + q.e) : "memory");
        }
      }
    }
    epi_sync();
    if (et == 0) mbar_arrive(&bars->done);
  }

  // ---------------- the pairs of each token added ----------------
  // A warp takes 128 features of one token, a lane four of them: the parts of
  // a choice in order, then its weight times their sum.  The reads of sixteen
  // parts go through shared memory (the stages are done with), so that they are
  // all under way in a loop of few instructions: unrolled for registers the
  // same code, run once and cold, took 3 us more.
  if (warp >= kEpi0 && units > 0) {
    bool ok = wait_or_abort(&bars->done, 0, limit, abort_flag, g.status) &&
              wait_or_abort(&bars->weights, 0, limit, abort_flag, g.status);
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    constexpr int kWarps = kThreads / 32 - kEpi0;
    const int terms = m.k * g.parts;
    float4* mine = reinterpret_cast<float4*>(smem + (warp - kEpi0) * 16 * 512) + lane;
    for (int c = (warp - kEpi0) * gridDim.x + blockIdx.x; ok && c < g.tb * m.T; c += gridDim.x * kWarps) {
      const int tk = c / g.tb, tile = c - tk * g.tb;
      // Every expert's parts of this tile have to be in y.
      if (lane == 0) {
        long long i = 0;
        while (ld_acquire(g.tickets + tile) < active * g.parts && i < limit) {
          if ((++i & 255) == 0 && *abort_flag) i = limit;
          __nanosleep(32);
        }
        if (i >= limit) {
          *abort_flag = 1;
          if (g.status) atomicExch(g.status, (int)DETFFN_ERR_TIMEOUT);
          ok = false;
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      __syncwarp();   // (lane 0's acquire comes before the reads of all)
      if (!ok) continue;
      const long long r = tile * 128ll + 4 * lane;
      const float* y = g.y + min(r, m.H - 4);   // (lanes past the last feature read the last and write nothing)
      // The choices whose h the two terms do not hold.  (Released with `ready`,
      // which the down units that were waited for have acquired.)
      unsigned again = 0;
      if constexpr (DT == DETFFN_F16)
        again = __ballot_sync(0xffffffffu, lane < m.k && !Terms<DT>::hold(__ldcg(g.top + t.pos[tk * m.k + min(lane, m.k - 1)])));
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f), one = s;
      int j = tk * m.k, part = 0;      // of the next read
      int ja = j, parta = 0;           // of the next addition
      for (int i0 = 0; i0 < terms; i0 += 16) {
        const int n = min(16, terms - i0);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(mine + i * 32)),
                       "l"(y + ((long long)part * P + t.pos[j]) * m.H)
                       : "memory");
          if (++part == g.parts) {
            part = 0;
            ++j;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const float4 v = mine[i * 32];
          one = parta == 0 ? v : make_float4(one.x + v.x, one.y + v.y, one.z + v.z, one.w + v.w);
          if (++parta == g.parts) {
            if constexpr (DT == DETFFN_F16) {
              if (again >> (ja - tk * m.k) & 1)
                one = down_rows<DT>(static_cast<const El*>(m.Wd) + (t.id[ja] * m.H + tile * 128ll) * m.I, g.h32 + t.pos[ja] * m.I,
                                    m.I, (int)min(128ll, m.H - tile * 128ll), lane);
            }
            const float w = t.w[ja];
            s = make_float4(fmaf(w, one.x, s.x), fmaf(w, one.y, s.y), fmaf(w, one.z, s.z), fmaf(w, one.w, s.w));
            parta = 0;
            ++ja;
          }
        }
      }
      if (r < m.H)
        *reinterpret_cast<uint2*>(static_cast<El*>(m.out) + tk * m.H + r) =
            make_uint2(Io<DT>::pair(s.x, s.y), Io<DT>::pair(s.z, s.w));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

template <int DT>
cudaError_t tensor(const MoeArgs& m, const MoeScratch& sc, const Waits& wt, int sm_count, cudaStream_t st) {
  static PerDevice ready;
  cudaError_t e =
      once_per_device(ready, [] { return cudaFuncSetAttribute(k_moe<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax); });
  if (e != cudaSuccess) return e;
  const bool f16 = DT == DETFFN_F16;
  CUtensorMap mWg, mWu, mWg32, mWu32, mWd, mX, mH[4];
  const long long dg[3] = {m.H, m.I, m.E}, dd[3] = {m.I, m.H, m.E}, dx[2] = {m.H, m.T}, dh[2] = {m.I, 2ll * m.T * m.k};
  const int bw[3] = {64, 64, 1}, bw32[3] = {64, 32, 1}, bx[2] = {64, (m.T + 15) / 16 * 16};
  if (!tc_make_map_nd(&mWg, f16, m.Wg, 3, dg, bw) || !tc_make_map_nd(&mWu, f16, m.Wu, 3, dg, bw) ||
      !tc_make_map_nd(&mWg32, f16, m.Wg, 3, dg, bw32) || !tc_make_map_nd(&mWu32, f16, m.Wu, 3, dg, bw32) ||
      !tc_make_map_nd(&mWd, f16, m.Wd, 3, dd, bw) || !tc_make_map_nd(&mX, f16, m.x, 2, dx, bx))
    return cudaErrorInvalidValue;
  // h by 8, 16, 32 or 64 rows: those that an expert of this call can take.
  for (int i = 0; i < 4; ++i) {
    const int bh[2] = {64, 8 << i};
    if (i > 0 && hrows(m.T) < 8 << i)
      mH[i] = mH[0];
    else if (!tc_make_map_nd(&mH[i], f16, m.h, 2, dh, bh))
      return cudaErrorInvalidValue;
  }
  Args g{};
  g.m = m;

  g.cols = 2 * hrows(m.T);
  const int xmost = 4 * ((m.T + 15) / 16 * 2048), hmost = 512 * hrows(m.T);
  const int stage = kWeightBytes + (xmost > hmost ? xmost : hmost);  // the largest
  const int rest = 1024 + (int)((sizeof(Bars) + 127) & ~127) + kXch + tables_bytes(m.E, m.T * m.k);
  g.ring = (kSmemMax - rest) & ~1023;
  if (g.ring < 2 * stage) return cudaErrorInvalidConfiguration;
  g.tb = (int)((m.H + 127) / 128);
  moe_parts(m.H, m.I, &g.parts, &g.kpart);
  g.claim = sc.counters;
  g.ready = sc.counters + 1;
  g.tickets = g.ready + m.E;
  g.y = sc.y;
  g.top = reinterpret_cast<unsigned*>(g.tickets + g.tb);
  g.h32 = sc.h32;
  g.status = wt.status;
  g.spin = wt.spin;
  g.stall = wt.stall;
  e = launch_moe_logits(m, sc.counters, 1 + m.E + g.tb + (f16 ? m.T * m.k : 0), st);
  if (e != cudaSuccess) return e;
  const long long most = (long long)(m.T * m.k < m.E ? m.T * m.k : m.E) * ((m.I + 31) / 32 + g.tb * g.parts);
  const int grid = (int)(most < sm_count ? most : sm_count);
  return launch_dependent(k_moe<DT>, dim3(grid), kThreads, kSmemMax, st, mWg, mWu, mWg32, mWu32, mWd, mX, mH[0], mH[1],
                          mH[2], mH[3], g);
}

}  // namespace

void moe_parts(long long H, long long I, int* parts, int* stages) {
  const int tiles = (int)((H + 127) / 128), kb = (int)((I + KS - 1) / KS);
  const int want = tiles < 16 ? 16 / tiles : 1;
  int per = (kb + want - 1) / want;
  if (per < 2) per = 2;
  *stages = per;
  *parts = (kb + per - 1) / per;
}

bool moe_tensor_covers(const MoeArgs& m) {
  const void* p[] = {m.x, m.Wg, m.Wu, m.Wd, m.h, m.out};
  for (const void* q : p)
    if ((uintptr_t)q & 15u) return false;
  return m.dtype != DETFFN_F32 && m.H % 8 == 0 && m.I % 8 == 0;
}

cudaError_t launch_moe_tensor(const MoeArgs& m, const MoeScratch& sc, const Waits& wt, int sm_count, cudaStream_t st) {
  return m.dtype == DETFFN_F16 ? tensor<DETFFN_F16>(m, sc, wt, sm_count, st)
                               : tensor<DETFFN_BF16>(m, sc, wt, sm_count, st);
}

}  // namespace detffn
