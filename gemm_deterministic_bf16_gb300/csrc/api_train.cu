// api_train.cu -- the C ABI of matrix products grouped by expert, products with
// 4-bit weights, and dropout.  Every call checks its arguments on the host
// before it launches anything, and allocates nothing.
#include <math.h>

#include <initializer_list>

#include "checks.h"
#include "dropout.h"
#include "grouped.h"
#include "w4.h"

using namespace detffn;

namespace {

// A matrix of contiguous rows at least `width` apart.
detffn_status matrix(const void* p, long long ld, long long rows, long long width, long long es) {
  if (!p) return DETFFN_ERR_INVALID_ARG;
  if (!on(p, es)) return DETFFN_ERR_ALIGN;
  if (rows > 1 && ld < width) return DETFFN_ERR_SHAPE;
  return DETFFN_OK;
}

// ---------------------------------------------------------------------------
// Grouped products
// ---------------------------------------------------------------------------
detffn_status grouped_sizes(long long R, long long E, long long K, long long N, int dtype) {
  if (!good_type(dtype)) return DETFFN_ERR_INVALID_ARG;
  if (R < 0 || R > kGroupedMaxRows || E < 1 || E > kGroupedMaxExperts || K < 1 || K > kGroupedMaxWidth || N < 1 ||
      N > kGroupedMaxWidth)
    return DETFFN_ERR_SHAPE;
  return DETFFN_OK;
}

detffn_status grouped_options(const detffn_options* o) {
  if (o && (o->path < DETFFN_PATH_AUTO || o->path > DETFFN_PATH_TENSOR || o->spin_limit < 0 ||
            (o->flags & ~DETFFN_FLAG_TEST_STALL)))
    return DETFFN_ERR_INVALID_ARG;
  return DETFFN_OK;
}

// Runs f on the handle's device.
template <class F>
detffn_status on_device(detffn_handle h, F&& f) {
  int prev = 0;
  TRYCU(cudaGetDevice(&prev));
  if (prev != h->device) TRYCU(cudaSetDevice(h->device));
  const detffn_status s = f();
  if (prev != h->device) cudaSetDevice(prev);
  return s;
}

// Scratch: rows whose width is not a multiple of 8 laid out on 16-byte boundaries.
struct GroupedScratch {
  uint16_t *x = nullptr, *W = nullptr, *dout = nullptr;
};
GroupedScratch grouped_plan(Arena& w, long long R, long long E, long long K, long long N, int dtype) {
  GroupedScratch s;
  if (dtype == DETFFN_F32) return s;
  if (K % 8) {
    s.x = w.take<uint16_t>(R * grouped_pad(K));
    s.W = w.take<uint16_t>(E * N * grouped_pad(K));
  }
  if (N % 8) s.dout = w.take<uint16_t>(R * grouped_pad(N));
  return s;
}

Waits grouped_waits(detffn_handle h, const detffn_options* o) {
  Waits wt;
  wt.status = h->d_status;
  if (o) {
    wt.spin = o->spin_limit;
    wt.stall = (o->flags & DETFFN_FLAG_TEST_STALL) ? 1 : 0;
  }
  return wt;
}

// The products of `a` that `what` lists: on the tensor cores where the rows lie, or
// can be laid out, on 16-byte boundaries.
detffn_status run_grouped(detffn_handle h, const GroupedArgs& a, std::initializer_list<Grouped> what, void* ws,
                          const detffn_options* o, cudaStream_t st) {
  const int path = o ? o->path : DETFFN_PATH_AUTO;
  const double es = (double)bytes_of(a.dtype), flops = 2.0 * a.R * a.K * a.N;
  // (the weights of as many experts as the rows can reach; the host does not know how many they do)
  const double most = a.R > a.E ? a.E : (double)a.R;
  GroupedArgs t = a;   // as the tensor kernel is to read it
  Arena w(ws);
  const GroupedScratch s = grouped_plan(w, a.R, a.E, a.K, a.N, a.dtype);
  const Rows W{a.W, a.ldw};
  bool lay_x = false, lay_W = false, lay_d = false, tensor = path != DETFFN_PATH_EXACT && a.dtype != DETFFN_F32;
  for (Grouped g : what) {
    if (g != Grouped::kInput) lay_x |= !grouped_boundary(a.x, a.R);
    if (g != Grouped::kWeight) lay_W |= !grouped_boundary(W, a.E * a.N);
    if (g != Grouped::kForward) lay_d |= !grouped_boundary(a.dout, a.R);
  }
  tensor = tensor && (!lay_x || s.x) && (!lay_W || s.W) && (!lay_d || s.dout);
  if (path == DETFFN_PATH_TENSOR && !tensor) return DETFFN_ERR_UNSUPPORTED;
  if (tensor) {
    if (lay_x) t.x = Rows{s.x, grouped_pad(a.K)};
    if (lay_W) t.W = s.W, t.ldw = grouped_pad(a.K);
    if (lay_d) t.dout = Rows{s.dout, grouped_pad(a.N)};
    const double rows = (lay_x ? (double)a.R * a.K : 0.0) + (lay_W ? most * a.N * a.K : 0.0) + (lay_d ? (double)a.R * a.N : 0.0);
    if (rows > 0.0)
      TRY(timed(h, st, "grouped_rows", 2.0 * es * rows, 0.0, [&]() -> detffn_status {
        if (lay_x) TRYCU(launch_grouped_rows(a.x, a.R, a.K, s.x, h->sm_count, st));
        if (lay_W) TRYCU(launch_grouped_matrices(a, s.W, h->sm_count, st));
        if (lay_d) TRYCU(launch_grouped_rows(a.dout, a.R, a.N, s.dout, h->sm_count, st));
        return DETFFN_OK;
      }, (lay_x ? 1 : 0) + (lay_W ? 1 : 0) + (lay_d ? 1 : 0)));
  }
  const Waits wt = grouped_waits(h, o);
  for (Grouped g : what)
    TRY(timed(h, st, tensor ? "grouped_tensor" : "grouped_general",
              es * ((double)a.R * (a.K + a.N) + (g == Grouped::kWeight ? a.E : most) * a.K * a.N), flops, [&] {
                return cu(tensor ? launch_grouped_tensor(t, g, wt, h->sm_count, st)
                                 : launch_grouped_general(a, g, h->sm_count, st));
              }));
  return DETFFN_OK;
}

// ---------------------------------------------------------------------------
// 4-bit weights
// ---------------------------------------------------------------------------
bool w4_group(int g) { return g == 32 || g == 64 || g == 128; }
long long w4_code_bytes(long long N, long long K) { return N * ((K + kW4Run - 1) / kW4Run) * (kW4Run / 2); }
long long w4_scale_bytes(long long N, long long K, int group, int type) { return N * ((K + group - 1) / group) * bytes_of(type); }

detffn_status w4_sizes(long long N, long long K, int group, int dtype, int stype) {
  if (!good_type(dtype) || !good_type(stype)) return DETFFN_ERR_INVALID_ARG;
  if (!w4_group(group)) return DETFFN_ERR_UNSUPPORTED;
  if (N < 1 || N > kW4MaxWidth || K < 1 || K > kW4MaxWidth) return DETFFN_ERR_SHAPE;
  return DETFFN_OK;
}
detffn_status w4_pointers(const void* codes, const void* scales) {
  if (!codes || !scales) return DETFFN_ERR_INVALID_ARG;
  return on(codes, 16) && on(scales, 4) ? DETFFN_OK : DETFFN_ERR_ALIGN;
}
// Rows as the kernels read them: where they are, or laid out at `to` by a launch of their own.
detffn_status w4_rows(const void* x, long long ldx, long long T, long long K, int dtype, void* to, int sms, cudaStream_t st,
                      W4Rows* r) {
  r->f16 = dtype == DETFFN_F16;
  if (dtype != DETFFN_F32 && w4_in_place(x, ldx, T, K)) {
    r->p = x;
    r->ld = T > 1 ? ldx : K;
    return DETFFN_OK;
  }
  r->p = to;
  r->ld = w4_pad(K);
  r->plane = T * r->ld;
  r->terms = dtype == DETFFN_F32 ? 3 : 1;
  return cu(launch_w4_rows(x, ldx, dtype, T, K, r->terms, to, sms, st));
}
W4Matrix w4_matrix(const void* codes, const void* scales, long long N, long long K, int group, int stype) {
  W4Matrix m;
  m.codes = static_cast<const uint8_t*>(codes);
  m.scales = scales;
  m.N = N;
  m.K = K;
  m.group = group;
  m.stype = stype;
  return m;
}

}  // namespace

extern "C" {

detffn_status detffn_grouped_workspace_size(long long R, long long E, long long K, long long N, int dtype, size_t* bytes) {
  if (!bytes) return DETFFN_ERR_INVALID_ARG;
  TRY(grouped_sizes(R, E, K, N, dtype));
  Arena w(nullptr);
  grouped_plan(w, R, E, K, N, dtype);
  *bytes = (w.off + 255) & ~(size_t)255;
  return DETFFN_OK;
}

detffn_status detffn_grouped_forward(detffn_handle h, const void* x, long long ldx, const void* W, const int* offsets,
                                     void* out, long long ldo, long long R, long long E, long long K, long long N,
                                     int dtype, void* ws, size_t ws_bytes, void* stream, const detffn_options* opts) {
  if (!h) return DETFFN_ERR_INVALID_ARG;
  TRY(grouped_sizes(R, E, K, N, dtype));
  TRY(grouped_options(opts));
  if (R == 0) return DETFFN_OK;
  const long long es = bytes_of(dtype);
  TRY(matrix(x, ldx, R, K, es));
  TRY(matrix(out, ldo, R, N, es));
  TRY(matrix(W, K, E * N, K, es));
  TRY(matrix(offsets, 1, E + 1, 1, 4));
  size_t need = 0;
  TRY(detffn_grouped_workspace_size(R, E, K, N, dtype, &need));
  if (need && (!ws || !on(ws, 256) || ws_bytes < need)) return DETFFN_ERR_WORKSPACE;
  const Span in[] = {rows_span(x, R, K, ldx, es), flat_span(W, E * N * K * es), flat_span(offsets, 4 * (E + 1))};
  const Span outs[] = {rows_span(out, R, N, ldo, es), flat_span(ws, (long long)need)};
  const int alias[] = {-1, -1};
  TRY(check_overlap(in, 3, outs, 2, alias));
  GroupedArgs a;
  a.R = R;
  a.K = K;
  a.N = N;
  a.E = (int)E;
  a.dtype = dtype;
  a.off = offsets;
  a.x = Rows{x, ldx};
  a.out = Rows{out, ldo};
  a.W = W;
  a.ldw = K;
  return on_device(h, [&] { return run_grouped(h, a, {Grouped::kForward}, ws, opts, (cudaStream_t)stream); });
}

detffn_status detffn_grouped_backward(detffn_handle h, const void* x, long long ldx, const void* W, const int* offsets,
                                      const void* dOut, long long lddo, void* dX, long long lddx, void* dW, long long R,
                                      long long E, long long K, long long N, int dtype, void* ws, size_t ws_bytes,
                                      void* stream, const detffn_options* opts) {
  if (!h) return DETFFN_ERR_INVALID_ARG;
  TRY(grouped_sizes(R, E, K, N, dtype));
  TRY(grouped_options(opts));
  if (!dX && !dW && R > 0) return DETFFN_ERR_INVALID_ARG;
  const long long es = bytes_of(dtype);
  cudaStream_t st = (cudaStream_t)stream;
  if (!on(dW, es)) return DETFFN_ERR_ALIGN;
  if (R == 0) {   // no rows: the weights' gradients are empty sums
    if (!dW) return DETFFN_OK;
    return on_device(h, [&] { return cu(cudaMemsetAsync(dW, 0, (size_t)(E * N * K * es), st)); });
  }
  TRY(matrix(dOut, lddo, R, N, es));
  TRY(matrix(offsets, 1, E + 1, 1, 4));
  if (dW) TRY(matrix(x, ldx, R, K, es));
  if (dX) TRY(matrix(W, K, E * N, K, es));
  if (dX) TRY(matrix(dX, lddx, R, K, es));
  size_t need = 0;
  TRY(detffn_grouped_workspace_size(R, E, K, N, dtype, &need));
  if (need && (!ws || !on(ws, 256) || ws_bytes < need)) return DETFFN_ERR_WORKSPACE;
  const Span in[] = {rows_span(dOut, R, N, lddo, es), rows_span(dW ? x : nullptr, R, K, ldx, es),
                     flat_span(dX ? W : nullptr, E * N * K * es), flat_span(offsets, 4 * (E + 1))};
  const Span outs[] = {rows_span(dX, R, K, lddx, es), flat_span(dW, E * N * K * es), flat_span(ws, (long long)need)};
  const int alias[] = {-1, -1, -1};
  TRY(check_overlap(in, 4, outs, 3, alias));
  GroupedArgs a;
  a.R = R;
  a.K = K;
  a.N = N;
  a.E = (int)E;
  a.dtype = dtype;
  a.off = offsets;
  a.x = Rows{x, ldx};
  a.W = W;
  a.ldw = K;
  a.dout = Rows{dOut, lddo};
  a.dx = Rows{dX, lddx};
  a.dW = dW;
  return on_device(h, [&]() -> detffn_status {
    if (dX && dW) return run_grouped(h, a, {Grouped::kInput, Grouped::kWeight}, ws, opts, st);
    return dX ? run_grouped(h, a, {Grouped::kInput}, ws, opts, st) : run_grouped(h, a, {Grouped::kWeight}, ws, opts, st);
  });
}

detffn_status detffn_w4_pack(const void* w, long long ldw, void* codes, void* scales, long long N, long long K, int group,
                             int dtype, int scale_dtype, void* stream) {
  TRY(w4_sizes(N, K, group, dtype, scale_dtype));
  TRY(w4_pointers(codes, scales));
  const long long es = bytes_of(dtype);
  TRY(matrix(w, ldw, N, K, es));
  const Span in[] = {rows_span(w, N, K, ldw, es)};
  const Span out[] = {flat_span(codes, w4_code_bytes(N, K)), flat_span(scales, w4_scale_bytes(N, K, group, scale_dtype))};
  const int alias[] = {-1, -1};
  TRY(check_overlap(in, 1, out, 2, alias));
  int sms = 0;
  TRY(current_sms(&sms));
  return cu(launch_w4_pack(w, ldw, dtype, w4_matrix(codes, scales, N, K, group, scale_dtype), sms, (cudaStream_t)stream));
}

detffn_status detffn_w4_unpack(const void* codes, const void* scales, void* w, long long ldw, long long N, long long K,
                               int group, int dtype, int scale_dtype, void* stream) {
  TRY(w4_sizes(N, K, group, dtype, scale_dtype));
  TRY(w4_pointers(codes, scales));
  const long long es = bytes_of(dtype);
  TRY(matrix(w, ldw, N, K, es));
  const Span in[] = {flat_span(codes, w4_code_bytes(N, K)), flat_span(scales, w4_scale_bytes(N, K, group, scale_dtype))};
  const Span out[] = {rows_span(w, N, K, ldw, es)};
  const int alias[] = {-1};
  TRY(check_overlap(in, 2, out, 1, alias));
  int sms = 0;
  TRY(current_sms(&sms));
  return cu(launch_w4_unpack(w4_matrix(codes, scales, N, K, group, scale_dtype), w, ldw, dtype, sms, (cudaStream_t)stream));
}

detffn_status detffn_w4_matvec_workspace_size(long long T, long long K, int dtype, size_t* bytes) {
  if (!bytes || !good_type(dtype)) return DETFFN_ERR_INVALID_ARG;
  if (T < 0 || T > kW4MaxTokens || K < 1 || K > kW4MaxWidth) return DETFFN_ERR_SHAPE;
  *bytes = (size_t)((dtype == DETFFN_F32 ? 3 : 1) * T * w4_pad(K) * 2 + 255) & ~(size_t)255;
  return DETFFN_OK;
}

detffn_status detffn_w4_matvec(const void* x, long long ldx, const void* codes, const void* scales, void* out,
                               long long ldo, long long T, long long N, long long K, int group, int dtype,
                               int scale_dtype, void* ws, size_t ws_bytes, void* stream) {
  TRY(w4_sizes(N, K, group, dtype, scale_dtype));
  size_t need = 0;
  TRY(detffn_w4_matvec_workspace_size(T, K, dtype, &need));
  if (T == 0) return DETFFN_OK;
  TRY(w4_pointers(codes, scales));
  const long long es = bytes_of(dtype);
  TRY(matrix(x, ldx, T, K, es));
  TRY(matrix(out, ldo, T, N, es));
  if (dtype != DETFFN_F32 && w4_in_place(x, ldx, T, K)) need = 0;
  if (need && (!ws || !on(ws, 256) || ws_bytes < need)) return DETFFN_ERR_WORKSPACE;
  const Span in[] = {rows_span(x, T, K, ldx, es), flat_span(codes, w4_code_bytes(N, K)),
                     flat_span(scales, w4_scale_bytes(N, K, group, scale_dtype))};
  const Span outs[] = {rows_span(out, T, N, ldo, es), flat_span(ws, (long long)need)};
  const int alias[] = {-1, -1};
  TRY(check_overlap(in, 3, outs, 2, alias));
  int sms = 0;
  TRY(current_sms(&sms));
  W4Args a;
  a.w = w4_matrix(codes, scales, N, K, group, scale_dtype);
  TRY(w4_rows(x, ldx, T, K, dtype, ws, sms, (cudaStream_t)stream, &a.x));
  a.out = out;
  a.ldo = ldo;
  a.T = (int)T;
  a.otype = dtype;
  return cu(launch_w4_matvec(a, sms, (cudaStream_t)stream));
}

detffn_status detffn_w4_workspace_size(long long T, long long H, long long I, int dtype, size_t* bytes) {
  size_t x = 0, h = 0;
  TRY(detffn_w4_matvec_workspace_size(T, H, dtype, &x));
  if (!bytes) return DETFFN_ERR_INVALID_ARG;
  TRY(detffn_w4_matvec_workspace_size(T, I, DETFFN_F32, &h));
  *bytes = x + h;
  return DETFFN_OK;
}

detffn_status detffn_w4_forward(const void* x, long long ldx, const void* gate_codes, const void* gate_scales,
                                const void* up_codes, const void* up_scales, const void* down_codes,
                                const void* down_scales, void* out, long long ldo, long long T, long long H, long long I,
                                int group, int dtype, int scale_dtype, void* ws, size_t ws_bytes, void* stream) {
  TRY(w4_sizes(I, H, group, dtype, scale_dtype));
  size_t need = 0, hbytes = 0;
  TRY(detffn_w4_workspace_size(T, H, I, dtype, &need));
  TRY(detffn_w4_matvec_workspace_size(T, I, DETFFN_F32, &hbytes));
  if (T == 0) return DETFFN_OK;
  TRY(w4_pointers(gate_codes, gate_scales));
  TRY(w4_pointers(up_codes, up_scales));
  TRY(w4_pointers(down_codes, down_scales));
  const long long es = bytes_of(dtype);
  TRY(matrix(x, ldx, T, H, es));
  TRY(matrix(out, ldo, T, H, es));
  if (!ws || !on(ws, 256) || ws_bytes < need) return DETFFN_ERR_WORKSPACE;
  const long long c1 = w4_code_bytes(I, H), s1 = w4_scale_bytes(I, H, group, scale_dtype), c2 = w4_code_bytes(H, I),
                  s2 = w4_scale_bytes(H, I, group, scale_dtype);
  const Span in[] = {rows_span(x, T, H, ldx, es), flat_span(gate_codes, c1), flat_span(gate_scales, s1),
                     flat_span(up_codes, c1),     flat_span(up_scales, s1),  flat_span(down_codes, c2),
                     flat_span(down_scales, s2)};
  const Span outs[] = {rows_span(out, T, H, ldo, es), flat_span(ws, (long long)need)};
  const int alias[] = {0, -1};   // (x is read before the last launch)
  TRY(check_overlap(in, 7, outs, 2, alias));
  int sms = 0;
  TRY(current_sms(&sms));
  cudaStream_t st = (cudaStream_t)stream;
  W4Args a;
  a.w = w4_matrix(gate_codes, gate_scales, I, H, group, scale_dtype);
  a.w2 = w4_matrix(up_codes, up_scales, I, H, group, scale_dtype);
  TRY(w4_rows(x, ldx, T, H, dtype, static_cast<char*>(ws) + hbytes, sms, st, &a.x));
  a.T = (int)T;
  // The hidden activation: terms planes of [T][I padded].
  a.out = ws;
  a.ldo = w4_pad(I);
  a.plane = T * w4_pad(I);
  a.terms = dtype == DETFFN_F32 ? 3 : 2;
  TRYCU(launch_w4_matvec(a, sms, st));
  W4Args d;
  d.w = w4_matrix(down_codes, down_scales, H, I, group, scale_dtype);
  d.x.p = ws;
  d.x.ld = a.ldo;
  d.x.plane = a.plane;
  d.x.terms = a.terms;
  d.T = (int)T;
  d.out = out;
  d.ldo = ldo;
  d.otype = dtype;
  return cu(launch_w4_matvec(d, sms, st));
}

detffn_status detffn_dropout_forward(const void* x, long long ldx, const void* residual, long long ldr, void* out,
                                     long long ldo, double p, unsigned long long seed, unsigned long long offset,
                                     const unsigned long long* state, long long M, long long H, int dtype, void* stream) {
  if (!good_type(dtype) || !(p >= 0.0 && p <= 1.0)) return DETFFN_ERR_INVALID_ARG;
  if (M < 0 || M > kMaxK || H < 1 || H > kMaxK) return DETFFN_ERR_SHAPE;
  if (M == 0) return DETFFN_OK;
  const long long es = bytes_of(dtype);
  TRY(matrix(x, ldx, M, H, es));
  TRY(matrix(out, ldo, M, H, es));
  if (residual) TRY(matrix(residual, ldr, M, H, es));
  if (!on(state, 8)) return DETFFN_ERR_ALIGN;
  // out may be exactly x or the residual: an element is read by the thread that writes it.
  const Span o = rows_span(out, M, H, ldo, es);
  const Span in[] = {rows_span(x, M, H, ldx, es), rows_span(residual, M, H, ldr, es), flat_span(state, 16)};
  for (int i = 0; i < 3; ++i)
    if (meet(o, in[i]) && !(i < 2 && same(o, in[i]))) return DETFFN_ERR_INVALID_ARG;
  DropoutArgs a;
  a.M = M;
  a.H = H;
  a.dtype = dtype;
  a.x = Rows{x, ldx};
  a.residual = Rows{residual, ldr};
  a.out = Rows{out, ldo};
  a.none = p >= 1.0;
  a.limit = a.none ? 0u : (uint32_t)floor(p * 4294967296.0);
  a.scale = a.none ? 0.0f : (float)(1.0 / (1.0 - p));
  a.seed = seed;
  a.offset = offset;
  a.state = state;
  int sms = 0;
  TRY(current_sms(&sms));
  return cu(launch_dropout(a, sms, (cudaStream_t)stream));
}

detffn_status detffn_dropout_backward(const void* dOut, long long lddo, void* dX, long long lddx, double p,
                                      unsigned long long seed, unsigned long long offset, const unsigned long long* state,
                                      long long M, long long H, int dtype, void* stream) {
  return detffn_dropout_forward(dOut, lddo, nullptr, 0, dX, lddx, p, seed, offset, state, M, H, dtype, stream);
}

}  // extern "C"
