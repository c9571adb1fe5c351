// k_join_ring.cuh -- the residual join over many rows of whole 16-byte vectors
// (the formulas are those of k_join.cuh).
//
// A CTA per SM holds groups of threads, one row at a time to a group and
// eight features (a unit) to a thread.  What bounds these passes is HBM, and
// what keeps it busy is bytes in flight: each group keeps a ring of rows in
// shared memory, filled by 1-D bulk copies several rows ahead, so that the
// loads of later rows run under the two sums of the current one.  The
// parameters stay in registers for all rows of a group, and in the backward
// pass so do the column sums.
#pragma once

#include "k_join.cuh"
#include "ptx.cuh"

namespace detffn {
namespace join {

constexpr int kRingBytes = 208 * 1024;   // shared memory for rows
constexpr int kRingMaxStages = 8;
constexpr int kRingMaxGroups = 16;       // 512 threads; groups of several warps (at most 8) have a named barrier each
constexpr int kRingSets = 152;           // CTAs: column sums are taken per CTA, so not of the GPU at hand

struct RingPlan {
  int G = 0, R = 0, S = 0, grid = 0;     // threads of a group, groups of a CTA, rows of a ring, CTAs
  int n = 0;                             // tensors of a row
  int bytes[5] = {};                     // their row bytes
  const unsigned char* p[5] = {};
  long long step[5] = {};                // bytes between rows
  int row = 0;                           // their sum
};

__device__ __forceinline__ void group_barrier(int group, int G) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(G) : "memory");
}

// Sums of N = 2 or 4 values over a group of G threads (whole warps, at most
// 16), the same in every thread, in an order fixed by G.  Stage one halves the
// values a lane carries with every exchange, so that lane l ends with the
// warp's sum of value l % N; stage two adds the warps the same way.  `buf`:
// [2][16 N] floats.  One barrier; one warp alone: none but __syncwarp.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], float* buf, int& turn, int G, int group, int t) {
  static_assert(N == 2 || N == 4, "");
  const int lane = t & 31;
  const bool odd = lane & 1, high = lane & 2;
  float x = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
  if (N == 4) {
    const float c = v[N - 2], d = v[N - 1];
    const float y = (odd ? d : c) + __shfl_xor_sync(0xffffffffu, odd ? c : d, 1);
    x = (high ? y : x) + __shfl_xor_sync(0xffffffffu, high ? x : y, 2);
  }
#pragma unroll
  for (int s = N; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  if (G > 32) {
    float* b = buf + turn * (16 * N);
    turn ^= 1;
    if (lane < N) b[(t >> 5) * N + lane] = x;
    group_barrier(group, G);
    const int n = (G >> 5) * N;
    x = lane < n ? b[lane] : 0.0f;
    if (N == 4) x += lane + 32 < n ? b[lane + 32] : 0.0f;
#pragma unroll
    for (int s = N; s < 32; s <<= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  } else {
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x, i);
}

// Where a group's rows live, and their arrival.
struct Ring1 {
  unsigned char* base;    // [S][row bytes]
  uint64_t* full;         // [S]
  int s = 0;
  uint32_t phase = 0;
};

// Issues the copies of row m into slot s (one thread).
__device__ __forceinline__ void ring_fill(const RingPlan& p, const Ring1& r, int s, long long m) {
  mbar_arrive_expect_tx(&r.full[s], (uint32_t)p.row);
  unsigned char* d = r.base + (size_t)s * p.row;
#pragma unroll
  for (int i = 0; i < 5; ++i)
    if (i < p.n) {
      bulk_g2s(d, p.p[i] + m * p.step[i], (uint32_t)p.bytes[i], &r.full[s]);
      d += p.bytes[i];
    }
}

// Waits for the row in the current slot.  Its copies were issued by this very
// group, so the wait ends; it is bounded all the same, and a row that never
// came would read as NaN.
__device__ __forceinline__ bool ring_wait(const Ring1& r) {
  return mbar_wait(&r.full[r.s], r.phase, kDefaultSpin, nullptr);
}

// Unit c / 8 of a row.
template <int DT>
__device__ __forceinline__ void unit(const void* row, int c, float (&v)[8]) {
  Io<DT>::ld8(static_cast<const typename Io<DT>::E*>(row) + c, v);
}
// The same of a parameter, in the rows' type or FP32; `fill` where there is none.
template <int DT>
__device__ __forceinline__ void param_unit(const void* p, int pdtype, int c, float fill, float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fill;
  } else if (DT == DETFFN_F32 || pdtype == DT) {
    unit<DT>(p, c, v);
  } else {
    unit<DETFFN_F32>(p, c, v);
  }
}
__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
  float s = a[0] * b[0], q = a[1] * b[1];
#pragma unroll
  for (int j = 2; j < 8; j += 2) s = fmaf(a[j], b[j], s), q = fmaf(a[j + 1], b[j + 1], q);
  return s + q;
}

// One sum and one barrier a row: the sum over z of the next row is taken
// together with the sum over out of this one.  A slot's row is read twice,
// once for each, and its slot is free after the barrier of the second.
//
// Forward.  V units to a thread: two where a row of units fills two warps, which
// halves what a row costs beside its elements.  PLAIN: both norms, and a gate
// (if any) that is the same for every row.
template <int DT, int V, bool PLAIN>
__global__ void __launch_bounds__(512, 1) k_fwd_ring(const __grid_constant__ JoinArgs a, const __grid_constant__ RingPlan p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t full[kRingMaxGroups * kRingMaxStages];
  __shared__ float sums[8 * 64];   // (groups of several warps: at most 8)
  using E = typename Io<DT>::E;
  const int G = p.G, group = threadIdx.x / G, t = threadIdx.x - group * G, H = a.H, rb = H * Io<DT>::kBytes;
  const bool has_z = PLAIN || a.z.p, has_post = PLAIN || a.w_post, has_pre = PLAIN || a.w_pre;
  const bool by_row = !PLAIN && a.gate && a.gate_rs;
  bool on[V];
  int c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {   // (threads past the row's end read its last unit and count for nothing)
    on[i] = 8 * (i * G + t) < H;
    c[i] = on[i] ? 8 * (i * G + t) : H - 8;
  }
  const long long first = (long long)blockIdx.x * p.R + group, step = (long long)gridDim.x * p.R;
  Ring1 ring{smem + (size_t)group * p.S * p.row, full + group * p.S};
  float* buf = sums + (G == 32 ? 0 : group * 64);
  if (t == 0) {
    for (int s = 0; s < p.S; ++s) mbar_init(&ring.full[s], 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  grid_dep_launch();
  if (t == 0)
    for (int s = 0; s < p.S; ++s)
      if (first + s * step < a.M) ring_fill(p, ring, s, first + s * step);
  float mix[V][8], pre[V][8];      // mix: scale * gate * w_post
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float w[8];
    param_unit<DT>(has_pre ? a.w_pre : nullptr, a.pdtype, c[i], 1.0f, pre[i]);
    param_unit<DT>(has_post ? a.w_post : nullptr, a.pdtype, c[i], 1.0f, w);
    param_unit<DT>(a.gate && a.gate_cs && !by_row ? a.gate : nullptr, a.pdtype, c[i],
                   a.gate && !a.gate_cs && !by_row ? param<DT>(a.gate, a.pdtype, 0) : 1.0f, mix[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) mix[i][j] *= a.scale * w[j];
  }
  const float inv = 1.0f / (float)H;
  int turn = 0;
  E* out = static_cast<E*>(const_cast<void*>(a.out.p)) + first * a.out.ld;
  E* y = static_cast<E*>(const_cast<void*>(a.y.p)) + first * a.y.ld;
  const long long out_step = step * a.out.ld, y_step = step * a.y.ld;
  __syncthreads();   // the barriers are initialised
  // The sum over z of the row in slot `s`.
  auto sum_z = [&](int s) {
    float v = 0.0f;
    if (has_post) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float n[8];
        unit<DT>(ring.base + (size_t)s * p.row + rb, c[i], n);
        v += on[i] ? dot8(n, n) : 0.0f;
      }
    }
    return v;
  };
  float sz = 0.0f;
  if (first < a.M) {
    const bool came = ring_wait(ring);
    float v[2] = {came ? sum_z(0) : __int_as_float(0x7fc00000), 0.0f};
    group_sums<2>(v, buf, turn, G, group, t);
    sz = v[0];
  }
  for (long long m = first; m < a.M; m += step, out += out_step, y += y_step) {
    const unsigned char* row = ring.base + (size_t)ring.s * p.row;
    const int slot = ring.s;
    if (++ring.s == p.S) {
      ring.s = 0;
      ring.phase ^= 1u;
    }
    float v[2] = {0.0f, 0.0f};
    if (m + step < a.M) v[0] = ring_wait(ring) ? sum_z(ring.s) : __int_as_float(0x7fc00000);
    float r[V][8];
    const float b = has_post ? rsqrtf(sz * inv + a.eps) : 1.0f;
    float g1 = 0.0f;
    if (by_row && !a.gate_cs) g1 = param<DT>(a.gate, a.pdtype, m * a.gate_rs);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unit<DT>(row, c[i], r[i]);
      if (has_z) {
        float n[8];
        unit<DT>(row + rb, c[i], n);
        if (by_row) {
          float g[8];
          param_unit<DT>(a.gate_cs ? row + 2 * rb : nullptr, a.pdtype, c[i], g1, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) n[j] *= g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = fmaf(b * n[j], mix[i][j], r[i][j]);
        if (on[i]) Io<DT>::st8(out + c[i], r[i]);
      }
      if (has_pre) v[1] += on[i] ? dot8(r[i], r[i]) : 0.0f;
    }
    group_sums<2>(v, buf, turn, G, group, t);
    if (t == 0 && m + p.S * step < a.M) ring_fill(p, ring, slot, m + p.S * step);
    sz = v[0];
    if (has_pre) {
      const float q = rsqrtf(v[1] * inv + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= q * pre[i][j];
        if (on[i]) Io<DT>::st8(y + c[i], r[i]);
      }
    }
  }
}

// Backward (rows of up to 4096 features, one unit to a thread).  PLAIN: both
// norms, dr given, and a gate (if any) that is the same for every row.
template <int DT, bool PLAIN>
__global__ void __launch_bounds__(512, 1) k_bwd_ring(const __grid_constant__ JoinArgs a, const __grid_constant__ RingPlan p) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t full[kRingMaxGroups * kRingMaxStages];
  __shared__ float sums[8 * (128 + 64)];   // (groups of several warps: at most 8)
  using E = typename Io<DT>::E;
  const int G = p.G, group = threadIdx.x / G, t = threadIdx.x - group * G, H = a.H, rb = H * Io<DT>::kBytes;
  const bool on = 8 * t < H;              // (threads past the row's end read its last unit and count for nothing)
  const int c = on ? 8 * t : H - 8;
  const long long first = (long long)blockIdx.x * p.R + group, step = (long long)gridDim.x * p.R;
  Ring1 ring{smem + (size_t)group * p.S * p.row, full + group * p.S};
  float *buf = sums + (G == 32 ? 0 : group * 192), *buf2 = buf + 128;
  if (t == 0) {
    for (int s = 0; s < p.S; ++s) mbar_init(&ring.full[s], 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  grid_dep_launch();
  if (t == 0)
    for (int s = 0; s < p.S; ++s)
      if (first + s * step < a.M) ring_fill(p, ring, s, first + s * step);
  const bool has_z = PLAIN || a.z.p, has_post = PLAIN || a.w_post, has_pre = PLAIN || a.w_pre, has_dr = PLAIN || a.dr.p;
  const bool feature = a.dgate && a.gate_cs && !a.gate_rs, scalar = a.dgate && !a.gate_cs && !a.gate_rs;
  const bool full_gate = !PLAIN && a.dgate && a.gate_cs && a.gate_rs, token = !PLAIN && a.dgate && !a.gate_cs && a.gate_rs;
  // Row layout: z, r, dy, dr, gate, those that there are.
  const int orr = has_z ? rb : 0, ody = orr + (has_pre ? rb : 0), odr = ody + (has_pre ? rb : 0), og = odr + (has_dr ? rb : 0);
  float pre[8], post[8], sg[8];   // w_pre, w_post, scale * gate
  param_unit<DT>(has_pre ? a.w_pre : nullptr, a.pdtype, c, 1.0f, pre);
  param_unit<DT>(has_post ? a.w_post : nullptr, a.pdtype, c, 1.0f, post);
  param_unit<DT>(feature ? a.gate : nullptr, a.pdtype, c, scalar ? param<DT>(a.gate, a.pdtype, 0) : 1.0f, sg);
  float apre[8], apost[8], agate[8];   // this thread's columns of the sums over tokens
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sg[j] *= a.scale;
    apre[j] = apost[j] = agate[j] = 0.0f;
  }
  const float inv = 1.0f / (float)H;
  int turn = 0, turn2 = 0;
  E* dxp = static_cast<E*>(const_cast<void*>(a.dx.p)) + first * a.dx.ld + c;
  E* dzp = static_cast<E*>(const_cast<void*>(a.dz.p)) + first * a.dz.ld + c;
  const long long dx_step = step * a.dx.ld, dz_step = step * a.dz.ld;
  __syncthreads();   // the barriers are initialised
  // Of the row in slot s: sum r^2, sum dy w_pre r, sum z^2.
  auto row_sums = [&](int s, float (&v)[4]) {
    const unsigned char* row = ring.base + (size_t)s * p.row;
    float x[8], w[8];
    if (has_pre) {
      unit<DT>(row + orr, c, x);
      unit<DT>(row + ody, c, w);
      v[0] = dot8(x, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= pre[j];
      v[1] = dot8(x, w);
    }
    if (has_post) {
      unit<DT>(row, c, x);
      v[2] = dot8(x, x);
    }
    if (!on) v[0] = v[1] = v[2] = 0.0f;
  };
  float s[3] = {0.0f, 0.0f, 0.0f};
  if (first < a.M) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (ring_wait(ring)) row_sums(0, v);
    else v[0] = v[2] = __int_as_float(0x7fc00000);
    group_sums<4>(v, buf, turn, G, group, t);
    s[0] = v[0], s[1] = v[1], s[2] = v[2];
  }
  for (long long m = first; m < a.M; m += step, dxp += dx_step, dzp += dz_step) {
    const unsigned char* row = ring.base + (size_t)ring.s * p.row;
    const int slot = ring.s;
    if (++ring.s == p.S) {
      ring.s = 0;
      ring.phase ^= 1u;
    }
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (m + step < a.M) {
      if (ring_wait(ring)) row_sums(ring.s, v);
      else v[0] = v[2] = __int_as_float(0x7fc00000);
    }
    // dx
    float d[8], z[8], x[8];
    if (has_dr) {
      unit<DT>(row + odr, c, d);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = 0.0f;
    }
    if (has_pre) {
      float dy[8];
      unit<DT>(row + orr, c, x);
      unit<DT>(row + ody, c, dy);
      const float q = rsqrtf(s[0] * inv + a.eps), k = s[1] * inv * (q * q * q);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float qd = q * dy[j];
        d[j] = fmaf(qd, pre[j], fmaf(-k, x[j], d[j]));
        apre[j] = fmaf(qd, x[j], apre[j]);
      }
      if (on) Io<DT>::st8(dxp, d);
    }
    const float b = has_post ? rsqrtf(s[2] * inv + a.eps) : 1.0f;
    float tok[2] = {0.0f, 0.0f};   // sum dx n
    if (has_z) {
      unit<DT>(row, c, z);
      if (full_gate || token) {
        param_unit<DT>(full_gate ? row + og : nullptr, a.pdtype, c, token ? param<DT>(a.gate, a.pdtype, m * a.gate_rs) : 0.0f, sg);
#pragma unroll
        for (int j = 0; j < 8; ++j) sg[j] *= a.scale;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = d[j] * (z[j] * b);
        const float w = u * sg[j];
        apost[j] += w;
        v[3] = fmaf(w, post[j], v[3]);   // sum dn w_post z b
        x[j] = u * post[j];              // dx n
        agate[j] += x[j];
      }
      if (token) tok[0] = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
      if (!on) v[3] = tok[0] = 0.0f;
    }
    group_sums<4>(v, buf, turn, G, group, t);
    if (t == 0 && m + p.S * step < a.M) ring_fill(p, ring, slot, m + p.S * step);
    s[0] = v[0], s[1] = v[1], s[2] = v[2];
    if (!PLAIN && !a.dz.p) continue;
    if (full_gate) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= a.scale;
      if (on) {
        if (DT == DETFFN_F32 || a.pdtype == DT) Io<DT>::st8(static_cast<E*>(a.dgate) + m * H + c, x);
        else Io<DETFFN_F32>::st8(static_cast<float*>(a.dgate) + m * H + c, x);
      }
    }
    if (token) {
      group_sums<2>(tok, buf2, turn2, G, group, t);
      if (t == 0) put_param<DT>(a.dgate, a.pdtype, m, a.scale * tok[0]);
    }
    const float k = v[3] * inv * (b * b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      d[j] *= sg[j] * post[j];
      if (has_post) d[j] = fmaf(b, d[j], -k * z[j]);
    }
    if (on) Io<DT>::st8(dzp, d);
  }
  // The CTA's column sums: its groups' added in order (the rings are done
  // with, so their memory holds them).  Little code, as it runs once and cold:
  // unrolled per kind and group it took 3 us more.
  __syncthreads();
  float* all = reinterpret_cast<float*>(smem);
  const int kinds = (a.dw_post ? 1 : 0) + (a.dw_pre ? 1 : 0) + (feature ? 1 : 0);
  {
    int kind = 0;
    auto put = [&](const float (&v)[8], float scale) {
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = scale * v[j];
      if (p.R > 1) Io<DETFFN_F32>::st8(all + kind * 4096 + 8 * threadIdx.x, w);
      else if (on) Io<DETFFN_F32>::st8(a.part + ((long long)kind * gridDim.x + blockIdx.x) * H + c, w);
      ++kind;
    };
    if (a.dw_post) put(apost, 1.0f);
    if (a.dw_pre) put(apre, 1.0f);
    if (feature) put(agate, a.scale);
  }
  if (p.R > 1) {
    __syncthreads();
    float* part = a.part + (long long)blockIdx.x * H;
#pragma unroll 1
    for (int kind = 0; kind < kinds; ++kind, part += (long long)gridDim.x * H)
#pragma unroll 1
      for (int i = threadIdx.x; i < H; i += blockDim.x) {
        float v = 0.0f;
#pragma unroll 1
        for (int q = 0; q < p.R; ++q) v += all[kind * 4096 + q * G * 8 + i];
        part[i] = v;
      }
  }
  if (scalar) {
    // One number: every thread's columns, added by warp and then in order.
    const float v = warp_sum(!on ? 0.0f : ((agate[0] + agate[1]) + (agate[2] + agate[3])) +
                                              ((agate[4] + agate[5]) + (agate[6] + agate[7])));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) all[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      float w = 0.0f;
      for (int q = 0; q < (int)blockDim.x >> 5; ++q) w += all[q];
      a.part[(long long)kinds * gridDim.x * H + blockIdx.x] = a.scale * w;
    }
  }
}

// The ring's layout for rows of these tensors; false where fewer than two
// rows fit a group's ring.
template <int DT>
bool ring_plan(const JoinArgs& a, bool back, RingPlan* out) {
  RingPlan p;
  const int es = Io<DT>::kBytes, ps = a.pdtype == DETFFN_F32 ? 4 : 2, units = a.H / 8;
  const int V = back || units < 64 ? 1 : 2, threads = 512;
  p.G = ((units + V - 1) / V + 31) / 32 * 32;
  if (p.G > threads) return false;
  const bool full = a.gate && a.gate_cs && a.gate_rs;
  auto add = [&](const void* q, long long ld, int bytes) {
    p.p[p.n] = static_cast<const unsigned char*>(q);
    p.step[p.n] = ld;
    p.bytes[p.n] = bytes;
    p.row += bytes;
    if (bytes) ++p.n;
  };
  const Rows* rows[4] = {back ? &a.z : &a.x, back ? &a.r : &a.z, &a.dy, &a.dr};
  for (int i = 0; i < (back ? 4 : 2); ++i)
    if (rows[i]->p) add(rows[i]->p, rows[i]->ld * es, a.H * es);
  if (full) add(a.gate, a.gate_rs * ps, a.H * ps);
  for (int i = 0; i < p.n; ++i)
    if (p.bytes[i] % 16) return false;
  // Few rows go to as many CTAs as there are before two share one.
  p.R = threads / p.G;
  if (p.R > (a.M + kRingSets - 1) / kRingSets) p.R = (int)((a.M + kRingSets - 1) / kRingSets);
    p.S = kRingBytes / (p.R * p.row);
  if (p.S < 2) return false;
  if (p.S > kRingMaxStages) p.S = kRingMaxStages;
  const long long need = (a.M + p.R - 1) / p.R;
  p.grid = (int)(need < kRingSets ? need : kRingSets);
  *out = p;
  return true;
}

template <auto K>
cudaError_t ring_launch(const JoinArgs& a, const RingPlan& p, cudaStream_t st) {
  static const cudaError_t setup = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (setup != cudaSuccess) return setup;
  const int smem = p.R * p.S * p.row > 49152 ? p.R * p.S * p.row : 49152;   // (48 KB: the groups' column sums)
  return launch_dependent(K, dim3(p.grid), p.G * p.R, smem, st, a, p);
}

// Whether a forward pass takes the ring kernel: it wins once its rows hold
// about 4 MB (measured, BF16, H = 4096: 152 rows 3.3 us without and 3.7 us with
// it, 608 rows 7.9 and 5.4; H = 1024: 1216 rows 4.1 and 4.3, 4864 rows 14.0 and
// 11.3), and always where the other kernel would have several units to a thread
// (H = 8192, 8 rows: 4.1 and 4.0).  The backward pass takes it wherever a row
// fits: from one row on it is no slower (H = 1024, 32 rows: 5.7 us without, 5.0
// with it; 4864 rows 60.9 and 22.4).
inline bool ring_forward(const JoinArgs& a, const RingPlan& p) { return a.M * p.row >= 4 << 20 || a.H > 4096; }

template <int DT>
cudaError_t forward(const JoinArgs& a, cudaStream_t st) {
  int threads;
  const int v = pick(a.H, &threads);
  const bool vec = vectors<DT>(a);
  RingPlan p;
  if (vec && ring_plan<DT>(a, false, &p) && ring_forward(a, p)) {
    const bool plain = a.z.p && a.w_post && a.w_pre && !(a.gate && a.gate_rs);
    if (a.H >= 512) return plain ? ring_launch<k_fwd_ring<DT, 2, true>>(a, p, st) : ring_launch<k_fwd_ring<DT, 2, false>>(a, p, st);
    return plain ? ring_launch<k_fwd_ring<DT, 1, true>>(a, p, st) : ring_launch<k_fwd_ring<DT, 1, false>>(a, p, st);
  }
  const long long most = 152ll * 16;
  const dim3 grid((unsigned)(a.M < most ? a.M : most));
  auto go = [&](auto k) { return launch_dependent(k, grid, threads, 0, st, a); };
  switch (v) {
    case 1: return go(vec ? k_fwd<DT, 1, true> : k_fwd<DT, 1, false>);
    case 2: return go(vec ? k_fwd<DT, 2, true> : k_fwd<DT, 2, false>);
    case 4: return go(vec ? k_fwd<DT, 4, true> : k_fwd<DT, 4, false>);
    default: return go(vec ? k_fwd<DT, 8, true> : k_fwd<DT, 8, false>);
  }
}

template <int DT>
cudaError_t backward(const JoinArgs& a, cudaStream_t st) {
  int threads;
  const int v = pick(a.H, &threads);
  const bool vec = vectors<DT>(a);
  int sets = (int)(a.M < kJoinSets ? a.M : kJoinSets);
  RingPlan p;
  const bool ring = vec && ring_plan<DT>(a, true, &p);
  const bool plain = a.w_post && a.w_pre && a.dr.p && !(a.gate && a.gate_rs);
  if (ring) sets = p.grid;
  auto go = [&](auto k) { return launch_dependent(k, dim3(sets), threads, 0, st, a); };
  cudaError_t e;
  if (ring) e = plain ? ring_launch<k_bwd_ring<DT, true>>(a, p, st) : ring_launch<k_bwd_ring<DT, false>>(a, p, st);
  else switch (v) {
    case 1: e = go(vec ? k_bwd<DT, 1, true> : k_bwd<DT, 1, false>); break;
    case 2: e = go(vec ? k_bwd<DT, 2, true> : k_bwd<DT, 2, false>); break;
    case 4: e = go(vec ? k_bwd<DT, 4, true> : k_bwd<DT, 4, false>); break;
    default: e = go(vec ? k_bwd<DT, 8, true> : k_bwd<DT, 8, false>); break;
  }
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
    e = launch_dependent(k_sets<DT>, dim3(1), sets_threads(sets), 0, st, (const float*)a.part + (long long)n * sets * a.H, sets, 1ll,
                         a.dgate, (void*)nullptr, (void*)nullptr, 0ll, a.pdtype);
  return e;
}

}  // namespace join
}  // namespace detffn
