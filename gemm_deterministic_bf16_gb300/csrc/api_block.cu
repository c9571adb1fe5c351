// api_block.cu -- the C ABI of the operators around the FFN: the residual join
// with its norms, 8-bit activation checkpoints, the mixture-of-experts layer.
// Every call checks its arguments on the host before it launches anything,
// and allocates nothing.
#include <math.h>

#include "block.h"
#include "checks.h"
#include "moe.h"

using namespace detffn;

namespace {

detffn_status join_sizes(long long M, long long H, int dtype, int pdtype) {
  if (!good_type(dtype) || !good_type(pdtype)) return DETFFN_ERR_INVALID_ARG;
  if (pdtype != dtype && pdtype != DETFFN_F32) return DETFFN_ERR_UNSUPPORTED;
  if (M < 0 || M > kMaxK || H < 1 || H > kJoinMaxH) return DETFFN_ERR_SHAPE;
  return DETFFN_OK;
}

detffn_status join_gate(const void* gate, long long rs, long long cs, long long M, long long H) {
  if (!gate) return DETFFN_OK;
  if ((cs != 0 && cs != 1) || rs < 0) return DETFFN_ERR_INVALID_ARG;
  if (cs == 1 && rs != 0 && M > 1 && rs < H) return DETFFN_ERR_SHAPE;
  return DETFFN_OK;
}

// The kernels index rows with the row stride alone, so one row of a tensor
// may have any stride.
detffn_status join_rows(const void* p, long long ld, long long M, long long H, long long es) {
  if (!p) return DETFFN_OK;
  if (!on(p, es)) return DETFFN_ERR_ALIGN;
  if (M > 1 && ld < H) return DETFFN_ERR_SHAPE;
  return DETFFN_OK;
}

long long gate_items(long long rs, long long cs, long long M, long long H) { return (rs ? M : 1) * (cs ? H : 1); }
Span gate_span(const void* p, long long rs, long long cs, long long M, long long H, long long ps) {
  return Span{p, rs ? M : 1, (cs ? H : 1) * ps, rs ? rs * ps : ps};
}

cudaError_t run_join(const JoinArgs& a, bool back, cudaStream_t st) {
  if (a.dtype == DETFFN_F32) return back ? join_backward_f32(a, st) : join_forward_f32(a, st);
  if (a.dtype == DETFFN_F16) return back ? join_backward_f16(a, st) : join_forward_f16(a, st);
  return back ? join_backward_bf16(a, st) : join_forward_bf16(a, st);
}

detffn_status ckpt_check(long long M, long long I, int dtype, const void* gq, const void* gs, const void* uq,
                         const void* us) {
  if (!good_type(dtype)) return DETFFN_ERR_INVALID_ARG;
  if (M < 0 || M > kMaxK || I < 1 || I > kMaxK) return DETFFN_ERR_SHAPE;
  if (M == 0) return DETFFN_OK;  // empty tensors may have null addresses
  if (!gq || !gs || !uq || !us) return DETFFN_ERR_INVALID_ARG;
  if (!on(gs, 4) || !on(us, 4)) return DETFFN_ERR_ALIGN;
  return DETFFN_OK;
}

}  // namespace

extern "C" {

detffn_status detffn_join_forward(const void* x, long long ldx, const void* z, long long ldz, const void* w_post,
                                  const void* gate, long long gate_rs, long long gate_cs, float scale,
                                  const void* w_pre, float eps, void* out, long long ldo, void* y, long long ldy,
                                  long long M, long long H, int dtype, int param_dtype, void* stream) {
  TRY(join_sizes(M, H, dtype, param_dtype));
  if (!(eps >= 0.0f) || isinf(eps)) return DETFFN_ERR_INVALID_ARG;
  TRY(join_gate(gate, gate_rs, gate_cs, M, H));
  if (M == 0) return DETFFN_OK;
  if (!x || (!z && (w_post || gate || out)) || (z && !out) || (!w_pre != !y) || (!z && !w_pre))
    return DETFFN_ERR_INVALID_ARG;
  const long long es = bytes_of(dtype), ps = bytes_of(param_dtype);
  TRY(join_rows(x, ldx, M, H, es));
  TRY(join_rows(z, ldz, M, H, es));
  TRY(join_rows(out, ldo, M, H, es));
  TRY(join_rows(y, ldy, M, H, es));
  if (!on(w_post, ps) || !on(w_pre, ps) || !on(gate, ps)) return DETFFN_ERR_ALIGN;
  const Span in[] = {rows_span(x, M, H, ldx, es), rows_span(z, M, H, ldz, es), flat_span(w_post, H * ps),
                     flat_span(w_pre, H * ps), gate_span(gate, gate_rs, gate_cs, M, H, ps)};
  const Span outs[] = {rows_span(out, M, H, ldo, es), rows_span(y, M, H, ldy, es)};
  const int alias[] = {0, -1};
  TRY(check_overlap(in, 5, outs, 2, alias));
  JoinArgs a;
  a.M = M;
  a.H = (int)H;
  a.dtype = dtype;
  a.pdtype = param_dtype;
  a.scale = scale;
  a.eps = eps;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.gate = gate;
  a.gate_rs = gate_rs;
  a.gate_cs = (int)gate_cs;
  a.x = Rows{x, ldx};
  a.z = Rows{z, ldz};
  a.out = Rows{out, ldo};
  a.y = Rows{y, ldy};
  return cu(run_join(a, false, (cudaStream_t)stream));
}

detffn_status detffn_join_workspace_size(long long M, long long H, size_t* bytes) {
  if (!bytes) return DETFFN_ERR_INVALID_ARG;
  if (M < 0 || M > kMaxK || H < 1 || H > kJoinMaxH) return DETFFN_ERR_SHAPE;
  const long long sets = M < kJoinSets ? M : kJoinSets;
  *bytes = (size_t)((3 * H + 1) * sets * 4 + 255) & ~(size_t)255;
  return DETFFN_OK;
}

detffn_status detffn_join_backward(const void* r, long long ldr, const void* dr, long long lddr, const void* dy,
                                   long long lddy, const void* z, long long ldz, const void* w_post, const void* gate,
                                   long long gate_rs, long long gate_cs, float scale, const void* w_pre, float eps,
                                   void* dx, long long lddx, void* dz, long long lddz, void* dgate, void* dw_post,
                                   void* dw_pre, long long M, long long H, int dtype, int param_dtype, void* ws,
                                   size_t ws_bytes, void* stream) {
  TRY(join_sizes(M, H, dtype, param_dtype));
  if (!(eps >= 0.0f) || isinf(eps)) return DETFFN_ERR_INVALID_ARG;
  TRY(join_gate(gate, gate_rs, gate_cs, M, H));
  const long long es = bytes_of(dtype), ps = bytes_of(param_dtype);
  cudaStream_t st = (cudaStream_t)stream;
  if ((!w_pre != !dw_pre) || (!w_post != !dw_post) || (!gate != !dgate) || (!w_pre && !dz && M > 0))
    return DETFFN_ERR_INVALID_ARG;
  if (!on(w_post, ps) || !on(w_pre, ps) || !on(gate, ps) || !on(dw_post, ps) || !on(dw_pre, ps) || !on(dgate, ps))
    return DETFFN_ERR_ALIGN;
  if (M == 0) {
    // No tokens: the parameters' gradients are empty sums.
    if (dw_pre) TRYCU(cudaMemsetAsync(dw_pre, 0, (size_t)(H * ps), st));
    if (dw_post) TRYCU(cudaMemsetAsync(dw_post, 0, (size_t)(H * ps), st));
    if (dgate && !gate_rs) TRYCU(cudaMemsetAsync(dgate, 0, (size_t)((gate_cs ? H : 1) * ps), st));
    return DETFFN_OK;
  }
  if ((w_pre && (!r || !dy || !dx)) || (!w_pre && (dy || dx)) || (!dr && !dy)) return DETFFN_ERR_INVALID_ARG;
  if ((!dz && (w_post || gate)) || ((w_post || gate) && !z)) return DETFFN_ERR_INVALID_ARG;
  TRY(join_rows(r, ldr, M, H, es));
  TRY(join_rows(dr, lddr, M, H, es));
  TRY(join_rows(dy, lddy, M, H, es));
  TRY(join_rows(z, ldz, M, H, es));
  TRY(join_rows(dx, lddx, M, H, es));
  TRY(join_rows(dz, lddz, M, H, es));
  size_t need = 0;
  TRY(detffn_join_workspace_size(M, H, &need));
  if (!ws || !on(ws, 256) || ws_bytes < need) return DETFFN_ERR_WORKSPACE;
  const Span in[] = {rows_span(dr, M, H, lddr, es), rows_span(z, M, H, ldz, es), rows_span(r, M, H, ldr, es),
                     rows_span(dy, M, H, lddy, es), flat_span(w_post, H * ps), flat_span(w_pre, H * ps),
                     gate_span(gate, gate_rs, gate_cs, M, H, ps)};
  const Span outs[] = {rows_span(dx, M, H, lddx, es), rows_span(dz, M, H, lddz, es), flat_span(dw_post, H * ps),
                       flat_span(dw_pre, H * ps), flat_span(dgate, gate_items(gate_rs, gate_cs, M, H) * ps),
                       flat_span(ws, (long long)need)};
  const int alias[] = {0, 1, -1, -1, -1, -1};
  TRY(check_overlap(in, 7, outs, 6, alias));
  JoinArgs a;
  a.M = M;
  a.H = (int)H;
  a.dtype = dtype;
  a.pdtype = param_dtype;
  a.scale = scale;
  a.eps = eps;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.gate = gate;
  a.gate_rs = gate_rs;
  a.gate_cs = (int)gate_cs;
  a.r = Rows{w_pre ? r : nullptr, ldr};
  a.dr = Rows{dr, lddr};
  a.dy = Rows{dy, lddy};
  a.z = Rows{w_post || gate ? z : nullptr, ldz};
  a.dx = Rows{dx, lddx};
  a.dz = Rows{dz, lddz};
  a.dgate = dgate;
  a.dw_post = dw_post;
  a.dw_pre = dw_pre;
  a.part = static_cast<float*>(ws);
  return cu(run_join(a, true, st));
}

detffn_status detffn_ckpt8_pack(const void* gate, const void* up, void* gate_codes, void* gate_scales, void* up_codes,
                                void* up_scales, long long M, long long I, int dtype, void* stream) {
  TRY(ckpt_check(M, I, dtype, gate_codes, gate_scales, up_codes, up_scales));
  if (M == 0) return DETFFN_OK;
  if (!gate || !up) return DETFFN_ERR_INVALID_ARG;
  const long long es = bytes_of(dtype), nb = (I + kCkptBlock - 1) / kCkptBlock;
  if (!on(gate, es) || !on(up, es)) return DETFFN_ERR_ALIGN;
  const Span in[] = {flat_span(gate, M * I * es), flat_span(up, M * I * es)};
  const Span out[] = {flat_span(gate_codes, M * I), flat_span(up_codes, M * I), flat_span(gate_scales, 4 * M * nb),
                      flat_span(up_scales, 4 * M * nb)};
  const int alias[] = {-1, -1, -1, -1};
  TRY(check_overlap(in, 2, out, 4, alias));
  CkptArgs a;
  a.M = M;
  a.I = I;
  a.dtype = dtype;
  a.gate = gate;
  a.up = up;
  a.gq = static_cast<int8_t*>(gate_codes);
  a.uq = static_cast<int8_t*>(up_codes);
  a.gs = static_cast<float*>(gate_scales);
  a.us = static_cast<float*>(up_scales);
  int sms = 0;
  TRY(current_sms(&sms));
  return cu(launch_ckpt8_pack(a, sms, (cudaStream_t)stream));
}

detffn_status detffn_ckpt8_unpack(const void* gate_codes, const void* gate_scales, const void* up_codes,
                                  const void* up_scales, void* gate, void* up, long long M, long long I, int dtype,
                                  void* stream) {
  TRY(ckpt_check(M, I, dtype, gate_codes, gate_scales, up_codes, up_scales));
  if (M == 0) return DETFFN_OK;
  if (!gate || !up) return DETFFN_ERR_INVALID_ARG;
  const long long es = bytes_of(dtype), nb = (I + kCkptBlock - 1) / kCkptBlock;
  if (!on(gate, es) || !on(up, es)) return DETFFN_ERR_ALIGN;
  const Span in[] = {flat_span(gate_codes, M * I), flat_span(up_codes, M * I), flat_span(gate_scales, 4 * M * nb),
                     flat_span(up_scales, 4 * M * nb)};
  const Span out[] = {flat_span(gate, M * I * es), flat_span(up, M * I * es)};
  const int alias[] = {-1, -1};
  TRY(check_overlap(in, 4, out, 2, alias));
  CkptArgs a;
  a.M = M;
  a.I = I;
  a.dtype = dtype;
  a.gate = gate;
  a.up = up;
  a.gq = static_cast<int8_t*>(const_cast<void*>(gate_codes));
  a.uq = static_cast<int8_t*>(const_cast<void*>(up_codes));
  a.gs = static_cast<float*>(const_cast<void*>(gate_scales));
  a.us = static_cast<float*>(const_cast<void*>(up_scales));
  int sms = 0;
  TRY(current_sms(&sms));
  return cu(launch_ckpt8_unpack(a, sms, (cudaStream_t)stream));
}

detffn_status detffn_ckpt8_silu_backward(const void* dh, const void* gate_codes, const void* gate_scales,
                                         const void* up_codes, const void* up_scales, void* dU, void* dG, void* h,
                                         long long M, long long I, int dtype, void* stream) {
  TRY(ckpt_check(M, I, dtype, gate_codes, gate_scales, up_codes, up_scales));
  if (M == 0) return DETFFN_OK;
  if (!dh || !dU || !dG) return DETFFN_ERR_INVALID_ARG;
  const long long es = bytes_of(dtype), nb = (I + kCkptBlock - 1) / kCkptBlock, n = M * I * es;
  if (!on(dh, es) || !on(dU, es) || !on(dG, es) || !on(h, es)) return DETFFN_ERR_ALIGN;
  const Span in[] = {flat_span(dh, n), flat_span(gate_codes, M * I), flat_span(up_codes, M * I),
                     flat_span(gate_scales, 4 * M * nb), flat_span(up_scales, 4 * M * nb)};
  const Span out[] = {flat_span(dU, n), flat_span(dG, n), flat_span(h, n)};
  const int alias[] = {-1, -1, -1};
  TRY(check_overlap(in, 5, out, 3, alias));
  CkptArgs a;
  a.M = M;
  a.I = I;
  a.dtype = dtype;
  a.dh = dh;
  a.gq = static_cast<int8_t*>(const_cast<void*>(gate_codes));
  a.uq = static_cast<int8_t*>(const_cast<void*>(up_codes));
  a.gs = static_cast<float*>(const_cast<void*>(gate_scales));
  a.us = static_cast<float*>(const_cast<void*>(up_scales));
  a.dU = dU;
  a.dG = dG;
  a.h = h;
  int sms = 0;
  TRY(current_sms(&sms));
  return cu(launch_ckpt8_silu_bwd(a, sms, (cudaStream_t)stream));
}

}  // extern "C"

namespace {

detffn_status moe_sizes(long long T, long long E, long long k, long long H, long long I, int dtype) {
  if (!good_type(dtype)) return DETFFN_ERR_INVALID_ARG;
  if (T < 0 || T > kMoeMaxTokens || E < 1 || E > kMoeMaxExperts || k < 1 || k > kMoeMaxTopK || k > E)
    return DETFFN_ERR_SHAPE;
  if (H < 1 || H > kMoeMaxWidth || I < 1 || I > kMoeMaxWidth) return DETFFN_ERR_SHAPE;
  return DETFFN_OK;
}

// Workspace layout; with experts and weights of their own where the caller
// takes none.
MoeArgs moe_plan(Arena& w, long long T, long long E, long long k, long long H, long long I, int dtype,
                 MoeScratch* sc) {
  MoeArgs a;
  a.T = (int)T;
  a.E = (int)E;
  a.k = (int)k;
  a.H = H;
  a.I = I;
  a.dtype = dtype;
  a.logits = w.take<float>(T * E);
  a.experts = w.take<int>(T * k);
  a.weights = w.take<float>(T * k);
  a.pos = w.take<int>(T * k);
  a.pair = w.take<int>(T * k);
  a.first = w.take<int>(E + 1);
  a.h = w.take<char>(T * k * I * 4);
  sc->counters = w.take<int>(1 + E + (H + 127) / 128 + T * k);
  int parts = 1, stages = 0;
  moe_parts(H, I, &parts, &stages);
  sc->y = w.take<float>(parts * T * k * H);
  // (FP16's, but a workspace sized for BF16 serves FP16 too)
  if (dtype != DETFFN_F32) sc->h32 = w.take<float>(T * k * I);
  return a;
}

}  // namespace

extern "C" {

detffn_status detffn_moe_workspace_size(long long T, long long E, int top_k, long long H, long long I, int dtype,
                                        size_t* bytes) {
  if (!bytes) return DETFFN_ERR_INVALID_ARG;
  TRY(moe_sizes(T, E, top_k, H, I, dtype));
  Arena w(nullptr);
  MoeScratch sc;
  moe_plan(w, T, E, top_k, H, I, dtype, &sc);
  *bytes = (w.off + 255) & ~(size_t)255;
  return DETFFN_OK;
}

detffn_status detffn_moe_forward(detffn_handle h, const void* x, const void* Wr, const void* Wg, const void* Wu,
                                 const void* Wd, void* out, int* experts, float* weights, long long T, long long E,
                                 int top_k, int normalize, long long H, long long I, int dtype, void* ws,
                                 size_t ws_bytes, void* stream, const detffn_options* opts) {
  if (!h) return DETFFN_ERR_INVALID_ARG;
  if (normalize != 0 && normalize != 1) return DETFFN_ERR_INVALID_ARG;
  TRY(moe_sizes(T, E, top_k, H, I, dtype));
  if (opts && (opts->path < DETFFN_PATH_AUTO || opts->path > DETFFN_PATH_TENSOR || opts->spin_limit < 0 ||
               (opts->flags & ~DETFFN_FLAG_TEST_STALL)))
    return DETFFN_ERR_INVALID_ARG;
  if (T == 0) return DETFFN_OK;
  if (!x || !Wr || !Wg || !Wu || !Wd || !out) return DETFFN_ERR_INVALID_ARG;
  const long long es = bytes_of(dtype);
  const void* ps[] = {x, Wr, Wg, Wu, Wd, out};
  for (const void* p : ps)
    if (!on(p, es)) return DETFFN_ERR_ALIGN;
  if (!on(experts, 4) || !on(weights, 4)) return DETFFN_ERR_ALIGN;
  size_t need = 0;
  TRY(detffn_moe_workspace_size(T, E, top_k, H, I, dtype, &need));
  if (!ws || !on(ws, 256) || ws_bytes < need) return DETFFN_ERR_WORKSPACE;
  const Span in[] = {flat_span(x, T * H * es), flat_span(Wr, E * H * es), flat_span(Wg, E * I * H * es),
                     flat_span(Wu, E * I * H * es), flat_span(Wd, E * I * H * es)};
  const Span outs[] = {flat_span(out, T * H * es), flat_span(experts, 4 * T * top_k), flat_span(weights, 4 * T * top_k),
                       flat_span(ws, (long long)need)};
  const int alias[] = {-1, -1, -1, -1};
  TRY(check_overlap(in, 5, outs, 4, alias));
  Arena w(ws);
  MoeScratch sc;
  MoeArgs a = moe_plan(w, T, E, top_k, H, I, dtype, &sc);
  a.x = x;
  a.Wr = Wr;
  a.Wg = Wg;
  a.Wu = Wu;
  a.Wd = Wd;
  a.out = out;
  a.normalize = normalize;
  if (experts) a.experts = experts;
  if (weights) a.weights = weights;
  const int path = opts ? opts->path : DETFFN_PATH_AUTO;
  const bool tensor = path != DETFFN_PATH_EXACT && moe_tensor_covers(a);
  if (path == DETFFN_PATH_TENSOR && !tensor) return DETFFN_ERR_UNSUPPORTED;
  Waits wt;
  wt.status = h->d_status;
  if (opts) {
    wt.spin = opts->spin_limit;
    wt.stall = (opts->flags & DETFFN_FLAG_TEST_STALL) ? 1 : 0;
  }
  int prev = 0;
  TRYCU(cudaGetDevice(&prev));
  if (prev != h->device) TRYCU(cudaSetDevice(h->device));
  // (the weights of as many experts as the pairs can reach; the host does not know how many they do)
  const double pairs = (double)T * top_k, hit = pairs < E ? pairs : E, width = 3.0 * H * I;
  const detffn_status s = timed(
      h, (cudaStream_t)stream, tensor ? "moe_tensor" : "moe_general", es * (2.0 * T * H + (double)E * H + hit * width),
      2.0 * T * E * H + 2.0 * pairs * width,
      [&] {
        return cu(tensor ? launch_moe_tensor(a, sc, wt, h->sm_count, (cudaStream_t)stream)
                         : launch_moe_general(a, sc, (cudaStream_t)stream));
      },
      tensor ? 2 : 5);
  if (prev != h->device) cudaSetDevice(prev);
  return s;
}

}  // extern "C"
