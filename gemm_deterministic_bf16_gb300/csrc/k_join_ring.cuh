// k_join_ring.cuh -- the residual join over many rows (the formulas are those
// of k_join.cuh).
//
// A CTA per SM holds groups of threads, one row at a time to a group and
// eight features (a unit) to a thread.  What bounds these passes is HBM, and
// what keeps it busy is bytes in flight: each group keeps a ring of rows in
// shared memory, filled by 1-D bulk copies several rows ahead, so that the
// loads of later rows run under the two sums of the current one.  The
// parameters stay in registers for all rows of a group, and in the backward
// pass so do the column sums.  Of the measured copy rate (6.69 TB/s) BF16 rows
// of 4096 features reach 85 % forward (16384 rows, 94.7 us) and 95 to 97 %
// backward (124 to 127 us).  Shorter rows are bound by what a row costs a warp
// beside its bytes (exchanges, a barrier, addresses: 389 instructions in all
// backward, with few warps to hide their latency): 16384 rows of 1024 features
// 80 % and 71 %, of 512 64 % and 57 %.
//
// VEC: rows of whole 16-byte vectors on 16-byte boundaries; a unit is eight
// features in a row.  Otherwise the copies take the 16-byte pieces that hold a
// byte of the row (a piece never crosses an allocation's boundary), and a unit
// is eight features 32 apart, a warp's 256 in a row, so that a warp's accesses
// to shared and global memory stay together wherever the row begins.  What
// bounds these is issue, an instruction or two for each element where a
// vector's eight share one (16384 x 1031: 36 us forward, 59 backward, 55 and 51 %
// of the copy rate).
#pragma once

#include <type_traits>

#include "k_join.cuh"
#include "ptx.cuh"

namespace detffn {
namespace join {

constexpr int kRingBytes = 208 * 1024;   // shared memory for rows
constexpr int kRingMaxStages = 8;
constexpr int kRingMaxGroups = 16;       // groups of several warps (at most 10) have a named barrier each
constexpr int kRingSets = kJoinSets;     // CTAs, whatever the GPU: column sums are taken per CTA

struct RingPlan {
  int G = 0, R = 0, S = 0, grid = 0;     // threads of a group, groups of a CTA, rows of a ring, CTAs
  int n = 0;                             // tensors of a row
  int es[5] = {};                        // their element bytes
  int off[5] = {};                       // where each lies in a slot
  const unsigned char* p[5] = {};
  long long step[5] = {};                // bytes between rows
  int row = 0;                           // bytes of a slot
  int per = 0, rest = 0;                 // rows of every group, and how many groups have one more
  int C = 1, width = 0;                  // CTAs that share a row, and the features of each but the last
};

// A group's ring of rows, in the order in which the group takes them.  Each
// tensor of a row is one lane's, which keeps its source and issues its copy: one
// thread for all took 170 instructions a row.
struct Ring1 {
  unsigned char *base, *at;        // [S][row bytes]; the slot of the next row to come
  uint64_t* full;                  // [S]
  int s = 0;                       // that slot
  uint32_t phase = 0;
  const unsigned char* src = nullptr;   // this lane's tensor: the next row to copy, from the CTA's first column on
  long long step = 0;              // bytes from it to the group's next row
  uint32_t off = 0, bytes = 0;     // where it lies in a slot; the bytes of its columns
};
// (Lanes t < p.n of the group's first warp copy.)
__device__ __forceinline__ void ring_init(const RingPlan& p, Ring1& r, int t, long long first, long long step, int col, int width) {
#pragma unroll
  for (int i = 0; i < 5; ++i)
    if (i == t && i < p.n) {
      r.src = p.p[i] + first * p.step[i] + (long long)col * p.es[i];
      r.step = step * p.step[i];
      r.off = (uint32_t)p.off[i];
      r.bytes = (uint32_t)(width * p.es[i]);
    }
  if (t == 0) {
    for (int s = 0; s < p.S; ++s) mbar_init(&r.full[s], (uint32_t)p.n);
    fence_mbar_init();
  }
}
// Issues the copy of the next row of this lane's tensor into slot s, at `slot`.
template <bool VEC>
__device__ __forceinline__ void ring_fill(Ring1& r, int s, unsigned char* slot) {
  const uintptr_t at = (uintptr_t)r.src;
  const uint32_t size = VEC ? r.bytes : (((uint32_t)at & 15u) + r.bytes + 15u) & ~15u;
  mbar_arrive_expect_tx(&r.full[s], size);
  bulk_g2s(slot + r.off, (const void*)(VEC ? at : at & ~(uintptr_t)15), size, &r.full[s]);
  r.src += r.step;
}
__device__ __forceinline__ void ring_next(const RingPlan& p, Ring1& r) {
  r.at += p.row;
  if (++r.s == p.S) {
    r.s = 0;
    r.at = r.base;
    r.phase ^= 1u;
  }
}

// Tensor i of a slot's row, which begins `off` bytes into the slot; rows that
// are not whole pieces begin 16-byte piece and a remainder further, which the
// address's low bits give: `low`, for the first row, and `step` more a row.
struct Part {
  uint32_t off, low, step;
};
template <bool VEC>
__device__ __forceinline__ Part part_of(const RingPlan& p, int i, long long first, long long step, int col) {
  Part r = {(uint32_t)p.off[i], 0, 0};
  if (!VEC) {
    r.low = (uint32_t)(uintptr_t)p.p[i] + (uint32_t)first * (uint32_t)p.step[i] + (uint32_t)(col * p.es[i]);
    r.step = (uint32_t)step * (uint32_t)p.step[i];
  }
  return r;
}
// The n-th row of the group.
template <bool VEC>
__device__ __forceinline__ const unsigned char* ring_row(const unsigned char* slot, const Part& p, uint32_t n) {
  return slot + p.off + (VEC ? 0u : (p.low + n * p.step) & 15u);
}

// Waits for the row in the current slot.  Its copies were issued by this very
// group, so the wait ends; it is bounded all the same, and what is formed from a
// row that never came is NaN.
__device__ __forceinline__ bool ring_wait(const Ring1& r) {
  return mbar_wait(&r.full[r.s], r.phase, kDefaultSpin, nullptr);
}

// What a pass has, when it is compiled for it (backward: z where it is read).  A
// pass compiled for any of it tests bits as it goes, and each test ends a run of
// instructions that the compiler can interleave: BF16, backward, 8192 x 4096, only
// the post-norm 73 us so and 47 compiled for it; only the pre-norm 86 and 57;
// both, 16384 x 2048, a gate per token 114 and 94, forward 57 and 53;
// forward, 16384 x 1031, 44 and 36.
enum Has : uint32_t { kZ = 1, kPost = 2, kPre = 4, kDr = 8, kDz = 16, kFull = 32, kToken = 64, kAny = 0 };

__host__ __device__ inline uint32_t has_of(const JoinArgs& a) {
  return (a.z.p ? kZ : 0u) | (a.w_post ? kPost : 0u) | (a.w_pre ? kPre : 0u) | (a.dr.p ? kDr : 0u) | (a.dz.p ? kDz : 0u) |
         (a.gate && a.gate_rs ? a.gate_cs ? kFull : kToken : 0u);
}

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums over the CTAs of a cluster: each CTA's four values (the same in all its
// threads) go to every CTA's shared memory, count there against a barrier of
// that CTA, and are added by rank.  `buf`: [2][8][4] floats; `bars`: one for each
// half, of one arrival.  Two halves are enough: a CTA sends exchange k + 2 only
// after every other has sent k + 1, and with it read k.  (With a barrier of the
// cluster instead 4864 x 8192 takes 146 us, and so 103.)
struct ClusterSums {
  float* buf;
  uint64_t* bars;
  int C, rank, half = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void operator()(float (&v)[4]) {
    float* b = buf + half * 32;
    uint64_t* bar = bars + half;
    if ((int)threadIdx.x < C) {
      if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, 16u * C);
      asm volatile(
          "{\n\t.reg .b32 a, m;\n\t"
          "mapa.shared::cluster.u32 a, %0, %2;\n\t"
          "mapa.shared::cluster.u32 m, %1, %2;\n\t"
          "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [a], {%3, %4, %5, %6}, [m];\n\t}" ::"r"(
              smem_u32(b + rank * 4)),
          "r"(smem_u32(bar)), "r"(threadIdx.x), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
          : "memory");
    }
    // Every CTA of the cluster has started and takes the same rows, so the wait
    // ends; it is bounded all the same, and sums that never came are NaN.
    bool came = false;
    for (long long i = 0; i < kDefaultSpin && !came; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(phase)
          : "memory");
      came = ok != 0;
    }
    float4 t = *reinterpret_cast<const float4*>(b);
    for (int r = 1; r < C; ++r) {
      const float4 o = *reinterpret_cast<const float4*>(b + r * 4);
      t.x += o.x, t.y += o.y, t.z += o.z, t.w += o.w;
    }
    const float none = __int_as_float(0x7fc00000);
    v[0] = came ? t.x : none;
    v[1] = came ? t.y : none;
    v[2] = came ? t.z : none;
    v[3] = came ? t.w : none;
    phase ^= (uint32_t)half;
    half ^= 1;
  }
};

// One sum and one barrier a row: the sum over z of the next row is taken
// together with the sum over out of this one.  A slot's row is read twice,
// once for each, and its slot is free after the barrier of the second.
//
// Forward.  V units to a thread: two where a row of units fills two warps, which
// halves what a row costs beside its elements.  WIDE: a cluster of CTAs shares
// each row of more than 8192 features, as in the backward pass.
template <int DT, int V, uint32_t HAS, bool VEC, bool WIDE = false>
__global__ void __launch_bounds__(512, 1) k_fwd_ring(const __grid_constant__ JoinArgs a, const __grid_constant__ RingPlan p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t full[kRingMaxGroups * kRingMaxStages];
  __shared__ float sums[8 * 80];   // (groups of several warps: at most 8)
  using E = typename Io<DT>::E;
  const int G = p.G, group = threadIdx.x / G, t = threadIdx.x - group * G, H = a.H;
  uint32_t has = HAS;
  if (HAS == kAny) {
    has = has_of(a);
    asm volatile("" : "+r"(has));   // (one register, so that a test is one instruction)
  }
  const bool has_z = has & kZ, has_post = has & kPost, has_pre = has & kPre, full_gate = has & kFull, token = has & kToken;
  const bool by_row = full_gate || token;
  int rank = 0;
  if (WIDE) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  __shared__ __align__(16) float across[2 * 8 * 4];
  __shared__ uint64_t crossed[2];
  ClusterSums cross{across, crossed, p.C, rank};
  if (WIDE && threadIdx.x == 0) {
    mbar_init(&crossed[0], 1);
    mbar_init(&crossed[1], 1);
  }
  const int col = rank * p.width, width = WIDE ? min(p.width, H - col) : H;
  Cols k[V];
#pragma unroll
  for (int i = 0; i < V; ++i) k[i] = cols_of<VEC>(i, G, t, width);
  const long long set = blockIdx.x / (WIDE ? p.C : 1), sets = gridDim.x / (WIDE ? p.C : 1);
  const long long first = set * p.R + group, step = sets * p.R;
  unsigned char* base = smem + group * p.S * p.row;
  Ring1 ring{base, base, full + group * p.S};
  GroupSums<2> sum2(sums + (G == 32 ? 0 : group * 80), G, group, t);
  ring_init(p, ring, t, first, step, col, width);
  __syncwarp();
  grid_dep_wait();
  grid_dep_launch();
  const int rows = p.per + (first < p.rest ? 1 : 0);   // of this group
  if (t < p.n)
    for (int s = 0; s < min(p.S, rows); ++s) ring_fill<VEC>(ring, s, base + s * p.row);
  const long long pcol = (long long)col * (a.pdtype == DETFFN_F32 ? 4 : 2);
  auto from = [&](const void* w) { return static_cast<const void*>(static_cast<const char*>(w) + pcol); };
  float mix[V][8], pre[V][8];      // mix: scale * gate * w_post
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float w[8];
    param_unit<DT, VEC>(has_pre ? from(a.w_pre) : nullptr, a.pdtype, k[i], 1.0f, pre[i]);
    param_unit<DT, VEC>(has_post ? from(a.w_post) : nullptr, a.pdtype, k[i], 1.0f, w);
    param_unit<DT, VEC>(a.gate && a.gate_cs && !by_row ? from(a.gate) : nullptr, a.pdtype, k[i],
                   a.gate && !a.gate_cs && !by_row ? param<DT>(a.gate, a.pdtype, 0) : 1.0f, mix[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) mix[i][j] *= a.scale * w[j];
  }
  const float inv = 1.0f / (float)H;
  // The parts of a row: x, z, gate.
  const Part px = part_of<VEC>(p, 0, first, step, col), pz = part_of<VEC>(p, 1, first, step, col),
             pg = part_of<VEC>(p, 2, first, step, col);
  E* out = static_cast<E*>(const_cast<void*>(a.out.p)) + first * a.out.ld + col;
  E* y = static_cast<E*>(const_cast<void*>(a.y.p)) + first * a.y.ld + col;
  const long long out_step = step * a.out.ld, y_step = step * a.y.ld;
  __syncthreads();   // the barriers are initialised
  if (WIDE) cluster_barrier();   // and every CTA of the cluster has started
  auto add = [&](float (&v)[2]) {
    sum2(v);
    if (WIDE) {
      float w[4] = {v[0], v[1], 0.0f, 0.0f};
      cross(w);
      v[0] = w[0], v[1] = w[1];
    }
  };
  auto all_rows = [&](const Cols (&k)[V]) __attribute__((always_inline)) {
    // The sum over z of the n-th row, in the next slot (0 where it is not wanted,
    // and NaN where the row never came: both reach every thread).
    auto sum_z = [&](int n) {
      float v = 0.0f;
      if (!ring_wait(ring)) return __int_as_float(0x7fc00000);
      if (has_post) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float z[8];
          unit<DT, VEC>(ring_row<VEC>(ring.at, pz, n), k[i], z);
          v += k[i].on ? dot8(z, z) : 0.0f;
        }
      }
      return v;
    };
    // A token's gate is read a row ahead.
    float sz = 0.0f, next_gate = by_row && !a.gate_cs && rows > 0 ? param<DT>(a.gate, a.pdtype, first * a.gate_rs) : 0.0f;
    if (rows > 0) {
      float v[2] = {sum_z(0), 0.0f};
      add(v);
      sz = v[0];
    }
    for (int n = 0; n < rows; ++n, out += out_step, y += y_step) {
      unsigned char* row = ring.at;
      const int slot = ring.s;
      ring_next(p, ring);
      float v[2] = {0.0f, 0.0f};
      if (n + 1 < rows) v[0] = sum_z(n + 1);
      float r[V][8];
      const float b = has_post ? rsqrtf(fmaf(sz, inv, a.eps)) : 1.0f + sz;
      const float g1 = next_gate;
      if (by_row && !a.gate_cs && n + 1 < rows) next_gate = param<DT>(a.gate, a.pdtype, (first + (n + 1) * step) * a.gate_rs);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        unit<DT, VEC>(ring_row<VEC>(row, px, n), k[i], r[i]);
        if (has_z) {
          float z[8];
          unit<DT, VEC>(ring_row<VEC>(row, pz, n), k[i], z);
          float g[8];
          if (by_row) param_unit<DT, VEC>(full_gate ? ring_row<VEC>(row, pg, n) : nullptr, a.pdtype, k[i], g1, g);
          // (gate * (scale * w_post) first, as it is for a gate that all rows share)
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i][j] = fmaf(b * z[j], by_row ? g[j] * mix[i][j] : mix[i][j], r[i][j]);
          put_unit<DT, VEC>(out, k[i], r[i]);
        }
        if (has_pre) v[1] += k[i].on ? dot8(r[i], r[i]) : 0.0f;
      }
      if (!has_z) v[1] += sz;
      add(v);
      if (t < p.n && n + p.S < rows) ring_fill<VEC>(ring, slot, row);
      sz = v[0];
      if (has_pre) {
        const float q = rsqrtf(fmaf(v[1], inv, a.eps));
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) r[i][j] *= q * pre[i][j];
          put_unit<DT, VEC>(y, k[i], r[i]);
        }
      }
    }
  };
  // (In rows that are not whole vectors all but the last warps have no feature
  // past the end, and are compiled for that.)
  bool whole = !VEC;
#pragma unroll
  for (int i = 0; i < V; ++i) whole = whole && __all_sync(0xffffffffu, k[i].on == 0xFFu);
  if (whole) {
    Cols w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = Cols{k[i].c, 0xFFu};
    all_rows(w);
  } else {
    all_rows(k);
  }
}

// Backward, one unit to a thread.  WIDE: a cluster of CTAs shares each row of
// more than 4096 features, a run of columns each, and the row's sums meet in
// shared memory across it.
//
// With n = b z, D = dx and c = scale gate w_post, a row needs sum D c n, and
// then dz = b D c - (sum D c n) b / H n.  The sums over tokens of dw_post and
// of a gate that is the same for every row have the factors scale gate and
// scale w_post of sum D n, so one accumulator serves both.  A row's r, dy and z
// are converted once and stay in registers over the barrier of its first sums.
template <int DT, uint32_t HAS, bool VEC, bool WIDE, int THREADS = 512>
__global__ void __launch_bounds__(THREADS, 1) k_bwd_ring(const __grid_constant__ JoinArgs a, const __grid_constant__ RingPlan p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t full[kRingMaxGroups * kRingMaxStages];
  __shared__ float sums[10 * 160];   // (groups of several warps: at most 10)
  using E = typename Io<DT>::E;
  const int G = p.G, group = threadIdx.x / G, t = threadIdx.x - group * G, H = a.H;
  int rank = 0;
  if (WIDE) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  __shared__ __align__(16) float across[2 * 8 * 4];
  __shared__ uint64_t crossed[2];
  ClusterSums cross{across, crossed, p.C, rank};
  if (WIDE && threadIdx.x == 0) {
    mbar_init(&crossed[0], 1);
    mbar_init(&crossed[1], 1);
  }
  const int col = rank * p.width, width = WIDE ? min(p.width, H - col) : H;
  const Cols cs = cols_of<VEC>(0, G, t, width);
  const bool on = cs.on != 0;
  const long long set = blockIdx.x / (WIDE ? p.C : 1), sets = gridDim.x / (WIDE ? p.C : 1);
  const long long first = set * p.R + group, step = sets * p.R;
  unsigned char* base = smem + group * p.S * p.row;
  Ring1 ring{base, base, full + group * p.S};
  GroupSums<4, THREADS> add(sums + (G == 32 ? 0 : group * 160), G, group, t);
  ring_init(p, ring, t, first, step, col, width);
  __syncwarp();
  grid_dep_wait();
  grid_dep_launch();
  const int rows = p.per + (first < p.rest ? 1 : 0);   // of this group
  if (t < p.n)
    for (int s = 0; s < min(p.S, rows); ++s) ring_fill<VEC>(ring, s, base + s * p.row);
  const bool uniform = a.dgate && !a.gate_rs;
  uint32_t has = HAS;
  if (HAS == kAny) {
    has = has_of(a);
    asm volatile("" : "+r"(has));   // (one register, so that a test is one instruction)
  }
  const bool has_z = has & kZ, has_post = has & kPost, has_pre = has & kPre, has_dr = has & kDr, has_dz = has & kDz;
  const bool full_gate = has & kFull, token = has & kToken;
  const bool by_row = full_gate || token, feature = uniform && a.gate_cs, scalar = uniform && !a.gate_cs;
  // The parts of a row: z, r, dy, dr, gate, those that there are.
  // (z is in a slot where it is given, whether it is read or not)
  const int ir = a.z.p != nullptr, idy = ir + has_pre, idr = idy + has_pre, ig = idr + has_dr;
  const Part pz = part_of<VEC>(p, 0, first, step, col), pr = part_of<VEC>(p, ir, first, step, col),
             pdy = part_of<VEC>(p, idy, first, step, col), pdr = part_of<VEC>(p, idr, first, step, col),
             pg = part_of<VEC>(p, ig, first, step, col);
  float pre[8], post[8], c[8];   // w_pre, w_post, scale * gate * w_post
  const long long pcol = (long long)col * (a.pdtype == DETFFN_F32 ? 4 : 2);
  auto from = [&](const void* q) { return static_cast<const void*>(static_cast<const char*>(q) + pcol); };
  param_unit<DT, VEC>(has_pre ? from(a.w_pre) : nullptr, a.pdtype, cs, 1.0f, pre);
  param_unit<DT, VEC>(has_post ? from(a.w_post) : nullptr, a.pdtype, cs, 1.0f, post);
  // scale * gate, the same for every row: wanted again at the end.
  auto gates = [&](float (&g)[8]) {
    param_unit<DT, VEC>(feature ? from(a.gate) : nullptr, a.pdtype, cs, scalar ? param<DT>(a.gate, a.pdtype, 0) : 1.0f, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= a.scale;
  };
  gates(c);
  float apre[8], apost[8];   // this thread's columns of the sums over tokens
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] *= post[j];
    apre[j] = apost[j] = 0.0f;
  }
  const float inv = 1.0f / (float)H;
  E* dxp = static_cast<E*>(const_cast<void*>(a.dx.p)) + first * a.dx.ld + col;
  E* dzp = static_cast<E*>(const_cast<void*>(a.dz.p)) + first * a.dz.ld + col;
  const long long dx_step = step * a.dx.ld, dz_step = step * a.dz.ld;
  __syncthreads();   // the barriers are initialised
  if (WIDE) cluster_barrier();   // and every CTA of the cluster has started
  auto sums4 = [&](float (&v)[4]) {
    add(v);
    if (WIDE) cross(v);
  };
  // The rows.  In rows that are not whole vectors all but the last warp have no
  // feature past the end, and are compiled for that.
  auto all_rows = [&](const Cols cs) __attribute__((always_inline)) {
    // The i-th row, in the next slot: r, dy, z, and sum r^2, sum dy w_pre r, sum z^2.
    float x[8], dy[8], n[8];
    auto arrive = [&](int i, float (&v)[4]) {
      const bool came = ring_wait(ring);
      if (has_pre) {
        unit<DT, VEC>(ring_row<VEC>(ring.at, pr, i), cs, x);
        unit<DT, VEC>(ring_row<VEC>(ring.at, pdy, i), cs, dy);
        v[0] = dot8(x, x);
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = dy[j] * pre[j];
        v[1] = dot8(x, w);
      }
      if (has_z) unit<DT, VEC>(ring_row<VEC>(ring.at, pz, i), cs, n);
      if (has_post) v[2] = dot8(n, n);
      if (VEC && !on) v[0] = v[1] = v[2] = 0.0f;
      if (!came) v[0] = v[2] = __int_as_float(0x7fc00000);
    };
    // A token's gate is read a row ahead.
    float next_gate = token && rows > 0 ? a.scale * param<DT>(a.gate, a.pdtype, first * a.gate_rs) : 1.0f;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (rows > 0) {
      arrive(0, s);
      sums4(s);
    }
    for (int i = 0; i < rows; ++i, dxp += dx_step, dzp += dz_step) {
      unsigned char* row = ring.at;
      const int slot = ring.s;
      ring_next(p, ring);
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d[8];
      if (has_dr) {
        unit<DT, VEC>(ring_row<VEC>(row, pdr, i), cs, d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = 0.0f;
      }
      if (has_pre) {
        // (in this order: q^3 alone leaves FP32's range for rows of 2e15 on)
        const float q = rsqrtf(fmaf(s[0], inv, a.eps)), k = s[1] * inv * q * q * q;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float qd = q * dy[j];
          d[j] = fmaf(qd, pre[j], fmaf(-k, x[j], d[j]));
          apre[j] = fmaf(qd, x[j], apre[j]);
        }
        put_unit<DT, VEC>(dxp, cs, d);
      }
      if (!has_pre && !has_post && s[2] != s[2]) {   // (the row never came; the norms' factors would show it)
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = s[2];
      }
      // d becomes D c, n is b z (without z: dz = scale dx).
      const float b = has_post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.0f;
      float bn[8];
      const float gate = next_gate;   // scale times a token's gate, or 1
      if (has_z) {
#pragma unroll
        for (int j = 0; j < 8; ++j) bn[j] = n[j] * b;
      }
      if (by_row) {
        const long long m = first + i * step;
        float g[8], u[8];
        if (token && i + 1 < rows) next_gate = a.scale * param<DT>(a.gate, a.pdtype, (m + step) * a.gate_rs);
        param_unit<DT, VEC>(full_gate ? ring_row<VEC>(row, pg, i) : nullptr, a.pdtype, cs, gate, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (full_gate) g[j] *= a.scale;
          u[j] = d[j] * bn[j];
          apost[j] = fmaf(u[j], g[j], apost[j]);
          u[j] *= post[j];
          d[j] *= g[j] * post[j];
        }
        if (token) {
          v[3] = ((u[0] + u[1]) + (u[2] + u[3])) + ((u[4] + u[5]) + (u[6] + u[7]));   // sum D n w_post: dgate's
        } else {
          v[3] = dot8(d, bn);
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] *= a.scale;
          if (DT == DETFFN_F32 || a.pdtype == DT) put_unit<DT, VEC>(static_cast<E*>(a.dgate) + m * H + col, cs, u);
          else put_unit<DETFFN_F32, VEC>(static_cast<float*>(a.dgate) + m * H + col, cs, u);
        }
      } else {
        if (has_z) {
#pragma unroll
          for (int j = 0; j < 8; ++j) apost[j] = fmaf(d[j], bn[j], apost[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= c[j];
        if (has_post) v[3] = dot8(d, bn);
      }
      if (VEC && !on) v[3] = 0.0f;
      // The next row's sums share this row's barrier.
      if (i + 1 < rows) arrive(i + 1, v);
      sums4(v);
      if (t < p.n && i + p.S < rows) ring_fill<VEC>(ring, slot, row);
      if (token && t == 0 && rank == 0) put_param<DT>(a.dgate, a.pdtype, first + i * step, a.scale * v[3]);
      if (has_post) {
        const float k = gate * v[3] * inv * b;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(b, d[j], -k * bn[j]);
      }
      if (has_dz) put_unit<DT, VEC>(dzp, cs, d);
      s[0] = v[0], s[1] = v[1], s[2] = v[2];
    }
  };
  if (!VEC && __all_sync(0xffffffffu, cs.on == 0xFFu)) all_rows(Cols{cs.c, 0xFFu});
  else all_rows(cs);
  // The CTA's column sums: its groups' added in order (the rings are done
  // with, so their memory holds them).  Little code, as it runs once and cold:
  // unrolled per kind and group it took 3 us more.
  __syncthreads();
  float* all = reinterpret_cast<float*>(smem);
  const int kinds = (a.dw_post ? 1 : 0) + (a.dw_pre ? 1 : 0) + (feature ? 1 : 0);
  {
    int kind = 0;
    auto put = [&](const float (&w)[8]) {
      // (a group's columns: G 8 floats, in their own order)
      if (p.R == 1) put_unit<DETFFN_F32, VEC>(a.part + (kind * sets + set) * H + col, cs, w);
      else put_unit<DETFFN_F32, VEC>(all + kind * 5120 + group * G * 8, cs, w);
      ++kind;
    };
    // (apost: sum dx n, and with a gate of each row sum dx n scale gate)
    float w[8];
    if (a.dw_post) {
      gates(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = by_row ? apost[j] : w[j] * apost[j];
      put(w);
    }
    if (a.dw_pre) put(apre);
#pragma unroll
    for (int j = 0; j < 8; ++j) apost[j] *= a.scale * post[j];
    if (feature) put(apost);
  }
  if (p.R > 1) {
    __syncthreads();
    float* part = a.part + set * H;
#pragma unroll 1
    for (int kind = 0; kind < kinds; ++kind, part += sets * H)
#pragma unroll 1
      for (int i = threadIdx.x; i < H; i += blockDim.x) {
        float v = 0.0f;
#pragma unroll 1
        for (int q = 0; q < p.R; ++q) v += all[kind * 5120 + q * G * 8 + i];
        part[i] = v;
      }
  }
  if (scalar) {
    // One number: every thread's columns, added by warp and then in order.
    const float v = warp_sum(!on ? 0.0f : ((apost[0] + apost[1]) + (apost[2] + apost[3])) +
                                              ((apost[4] + apost[5]) + (apost[6] + apost[7])));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) all[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      float w = 0.0f;
      for (int q = 0; q < (int)blockDim.x >> 5; ++q) w += all[q];
      a.part[kinds * sets * H + blockIdx.x] = w;
    }
  }
}

// The ring's layout for rows of these tensors; false where fewer than two
// rows fit a group's ring.  V: units to a thread.
template <int DT>
bool ring_plan(const JoinArgs& a, bool back, bool vec, int V, int threads, RingPlan* out) {
  RingPlan p;
  const int es = Io<DT>::kBytes, ps = a.pdtype == DETFFN_F32 ? 4 : 2;
  while (a.H > p.C * threads * 8 * V && p.C < 8) p.C *= 2;
  p.width = ((a.H + p.C - 1) / p.C + 7) / 8 * 8;
  const int units = p.width / 8;
  p.G = ((units + V - 1) / V + 31) / 32 * 32;
  if (p.G > threads) return false;
  const bool full = a.gate && a.gate_cs && a.gate_rs;
  auto add = [&](const void* q, long long step, int bytes) {
    p.p[p.n] = static_cast<const unsigned char*>(q);
    p.step[p.n] = step;
    p.es[p.n] = bytes;
    p.off[p.n++] = p.row;
    p.row += (p.width * bytes + 15) / 16 * 16 + (vec ? 0 : 16);
  };
  const Rows* rows[4] = {back ? &a.z : &a.x, back ? &a.r : &a.z, &a.dy, &a.dr};
  for (int i = 0; i < (back ? 4 : 2); ++i)
    if (rows[i]->p) add(rows[i]->p, rows[i]->ld * es, es);
  if (full) add(a.gate, a.gate_rs * ps, ps);
  // Few rows go to as many CTAs as there are before two share one.
  // (Clusters of four fit 36 times on this GPU's SMs, and of eight 15 times: with
  // 38 the last two wait for a second round, 2432 x 16384 198 us and 110 so.)
  const int most = p.C == 4 ? 36 : p.C == 8 ? 15 : kRingSets / p.C;
  p.R = p.C > 1 ? 1 : threads / p.G;
  if (p.R > kRingMaxGroups) p.R = kRingMaxGroups;
  if (p.R > (a.M + most - 1) / most) p.R = (int)((a.M + most - 1) / most);
  p.S = kRingBytes / (p.R * p.row);
  if (p.S < 2) return false;
  if (p.S > kRingMaxStages) p.S = kRingMaxStages;
  const long long need = (a.M + p.R - 1) / p.R;
  p.grid = (int)(need < most ? need : most) * p.C;
  p.per = (int)(a.M / ((long long)(p.grid / p.C) * p.R));
  p.rest = (int)(a.M % ((long long)(p.grid / p.C) * p.R));
  *out = p;
  return true;
}

template <auto K>
cudaError_t ring_launch(const JoinArgs& a, const RingPlan& p, cudaStream_t st) {
  static PerDevice ready;
  const cudaError_t e =
      once_per_device(ready, [] { return cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes); });
  if (e != cudaSuccess) return e;
  const int least = 3 * 5120 * 4;   // the groups' column sums
  const int smem = p.R * p.S * p.row > least ? p.R * p.S * p.row : least;
  return launch_cluster(K, dim3(p.grid), p.G * p.R, smem, p.C, st, a, p);
}

// Whether a forward pass takes the ring kernel: it wins once its rows hold some
// 4 to 7 MB (measured, BF16, H = 4096: 152 rows 3.1 us without and 3.6 us with it,
// 304 rows 3.9 and 4.2, 456 rows 6.3 and 5.3, 1216 rows 15.1 and 11.7; H = 1024: 1216
// rows 3.8 and 4.4, 2432 rows 6.6 and 5.5; H = 256: 8192 rows 5.0 and 5.0, 16384
// rows 11.3 and 9.2; FP32, H = 4096: even from 152 rows on), and takes what the other
// does not: rows of more than 4096 features and rows that are not whole vectors.
inline bool ring_forward(const JoinArgs& a, const RingPlan& p, bool vec) {
  return !vec || a.M * p.row >= 4 << 20 || a.H > 4096;
}

template <uint32_t H>
using Kind = std::integral_constant<uint32_t, H>;

template <int DT>
cudaError_t forward(const JoinArgs& a, cudaStream_t st) {
  const bool vec = vectors<DT>(a);
  RingPlan p;
  const bool two = vec ? a.H >= 512 : a.H > 4096;   // units to a thread
  if (!ring_plan<DT>(a, false, vec, two ? 2 : 1, 512, &p)) return cudaErrorInvalidConfiguration;   // (two rows always fit)
  if (ring_forward(a, p, vec)) {
    // The passes that are compiled for what they have: a unit to a thread of rows
    // that are not whole vectors and two of those that are, and else both norms
    // with a gate (if any) that is the same for every row.
    const uint32_t has = has_of(a);
    cudaError_t e = cudaErrorInvalidConfiguration;
    auto one = [&](auto h) {
      constexpr uint32_t HAS = decltype(h)::value;
      if (HAS != kAny && HAS != has) return false;
      if constexpr (HAS == kAny || HAS == (kPost | kPre | kZ)) {
        if (p.C > 1) {
          e = vec ? ring_launch<k_fwd_ring<DT, 2, HAS, true, true>>(a, p, st) : ring_launch<k_fwd_ring<DT, 2, HAS, false, true>>(a, p, st);
          return true;
        }
        if (two != vec) {
          e = vec ? ring_launch<k_fwd_ring<DT, 1, HAS, true>>(a, p, st) : ring_launch<k_fwd_ring<DT, 2, HAS, false>>(a, p, st);
          return true;
        }
      } else if (p.C > 1 || two != vec) {
        return false;
      }
      e = vec ? ring_launch<k_fwd_ring<DT, 2, HAS, true>>(a, p, st) : ring_launch<k_fwd_ring<DT, 1, HAS, false>>(a, p, st);
      return true;
    };
    auto any_of = [&](auto... h) { return (one(h) || ...); };
    any_of(Kind<kPost | kPre | kZ>{}, Kind<kPost | kPre | kZ | kToken>{}, Kind<kPost | kPre | kZ | kFull>{},
           Kind<kPost | kZ>{}, Kind<kPost | kZ | kToken>{}, Kind<kPost | kZ | kFull>{},
           Kind<kPre | kZ>{}, Kind<kPre | kZ | kToken>{}, Kind<kPre | kZ | kFull>{}, Kind<kPre>{}, Kind<kAny>{});
    return e;
  }
  // Few rows of whole vectors (a thread's two units go to two threads).
  const long long most = 152ll * 16;
  return launch_dependent(two ? k_fwd<DT, true> : k_fwd<DT, false>, dim3((unsigned)(a.M < most ? a.M : most)),
                          two ? 2 * p.G : p.G, 0, st, a);
}

// Whether a backward pass takes 640 threads instead of 512 to a CTA, and 96
// registers a thread instead of 128: with one norm its values fit, and a row of
// 5120 features needs no second CTA (BF16, the pre-norm alone, 8192 x 5120: 118 us
// with 512, 70 with 640; 8192 x 2560: 49 and 37; shorter rows even).  With z
// beside the pre-norm registers spill (16384 x 1024, a gate per feature: 36 and
// 49), which pays for rows of more than 4096 features alone (8192 x 5120, a gate
// per token: 150 and 118).  768 threads are slower (16384 x 1024: 33 and 41).
template <int DT>
bool one_norm(uint32_t has, int H) {
  if (DT == DETFFN_F32 || H > 5120 || !(has & kDr) || !(has & kDz)) return false;
  if ((has & kPre) && (has & kPost)) return false;
  if ((has & kPre) && (has & kZ)) return H > 4096;
  return (has & (kPre | kPost)) != 0;
}
template <int DT, uint32_t HAS>
cudaError_t wide_cta(const JoinArgs& a, const RingPlan& p, cudaStream_t st) {
  // (one_norm holds for no other pass)
  if constexpr (DT != DETFFN_F32 && HAS != kAny && !((HAS & kPre) && (HAS & kPost)))
    return ring_launch<k_bwd_ring<DT, HAS, true, false, 640>>(a, p, st);
  else return cudaErrorInvalidConfiguration;
}

template <int DT>
cudaError_t backward(const JoinArgs& a, cudaStream_t st) {
  const bool vec = vectors<DT>(a);
  RingPlan p;
  uint32_t has = has_of(a);
  if (!(has & kPost) && !a.dgate) has &= ~kZ;   // (z is not read)
  const int threads = vec && one_norm<DT>(has, a.H) ? 640 : 512;
  if (!ring_plan<DT>(a, true, vec, 1, threads, &p)) return cudaErrorInvalidConfiguration;   // (two rows always fit)
  const int sets = p.grid / p.C;
  // The passes that are compiled for what they have.
  cudaError_t e = cudaErrorInvalidConfiguration;
  auto one = [&](auto h) {
    constexpr uint32_t HAS = decltype(h)::value;
    if (HAS != kAny && HAS != has) return false;
    if (p.C > 1) e = vec ? ring_launch<k_bwd_ring<DT, HAS, true, true>>(a, p, st) : ring_launch<k_bwd_ring<DT, HAS, false, true>>(a, p, st);
    else if (threads > 512) e = wide_cta<DT, HAS>(a, p, st);
    else e = vec ? ring_launch<k_bwd_ring<DT, HAS, true, false>>(a, p, st) : ring_launch<k_bwd_ring<DT, HAS, false, false>>(a, p, st);
    return true;
  };
  constexpr uint32_t kBoth = kPost | kPre, kIn = kDr | kDz, kInZ = kIn | kZ;
  auto any_of = [&](auto... h) { return (one(h) || ...); };
  any_of(Kind<kBoth | kInZ>{}, Kind<kBoth | kInZ | kToken>{}, Kind<kBoth | kInZ | kFull>{},
         Kind<kPost | kInZ>{}, Kind<kPost | kInZ | kToken>{}, Kind<kPost | kInZ | kFull>{},
         Kind<kPre | kIn>{}, Kind<kPre | kInZ>{}, Kind<kPre | kInZ | kToken>{}, Kind<kPre | kInZ | kFull>{}, Kind<kAny>{});
  if (e != cudaSuccess) return e;
  void* out[3] = {};
  int n = 0;
  if (a.dw_post) out[n++] = a.dw_post;
  if (a.dw_pre) out[n++] = a.dw_pre;
  if (a.dgate && a.gate_cs && !a.gate_rs) out[n++] = a.dgate;
  if (n) {
    e = launch_dependent(k_sets<DT>, dim3((unsigned)((a.H + 31) / 32), n), sets_threads(sets), 0, st, (const float*)a.part, sets,
                         (long long)a.H, out[0], out[1], out[2], (long long)sets * a.H, a.pdtype);
    if (e != cudaSuccess) return e;
  }
  if (a.dgate && !a.gate_cs && !a.gate_rs)
    e = launch_dependent(k_sets<DT>, dim3(1), sets_threads(p.grid), 0, st, (const float*)a.part + (long long)n * sets * a.H, p.grid, 1ll,
                         a.dgate, (void*)nullptr, (void*)nullptr, 0ll, a.pdtype);
  return e;
}

}  // namespace join
}  // namespace detffn
