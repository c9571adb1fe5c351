// checks.h -- argument checks shared by the C entries that take operands of
// several types and strides: types, alignment, operands that share bytes.
#pragma once

#include "handle.h"

namespace detffn {

inline bool good_type(int t) { return t == DETFFN_F32 || t == DETFFN_F16 || t == DETFFN_BF16; }
inline long long bytes_of(int t) { return t == DETFFN_F32 ? 4 : 2; }
inline bool on(const void* p, long long n) { return ((uintptr_t)p % (uintptr_t)n) == 0; }

// One operand of a call, for the overlap checks: `rows` rows of `row` bytes,
// `step` bytes apart.
struct Span {
  const void* p = nullptr;
  long long rows = 0, row = 0, step = 0;
};

// Whether two operands share a byte.  Rows of equal step may interleave (the
// column halves of one buffer); otherwise their whole extents count.
inline bool meet(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.row <= 0 || b.row <= 0) return false;
  if (!overlap(a.p, (a.rows - 1) * a.step + a.row, b.p, (b.rows - 1) * b.step + b.row)) return false;
  if (a.rows > 1 && b.rows > 1 && a.step == b.step && a.step > 0) {
    const long long d = (long long)(((uintptr_t)b.p - (uintptr_t)a.p) % (uintptr_t)a.step);
    const long long up = (uintptr_t)b.p >= (uintptr_t)a.p
                             ? d
                             : (a.step - (long long)(((uintptr_t)a.p - (uintptr_t)b.p) % (uintptr_t)a.step)) % a.step;
    return !(up >= a.row && a.step - up >= b.row);
  }
  return true;
}

inline bool same(const Span& a, const Span& b) { return a.p == b.p && (a.step == b.step || a.rows <= 1); }

// Every output against every input and every other output.  Output `o` may be
// exactly input alias[o] (in place); -1: no input.
inline detffn_status check_overlap(const Span* in, int ni, const Span* out, int no, const int* alias) {
  for (int o = 0; o < no; ++o) {
    for (int i = 0; i < ni; ++i)
      if (meet(out[o], in[i]) && !(alias[o] == i && same(out[o], in[i]))) return DETFFN_ERR_INVALID_ARG;
    for (int q = o + 1; q < no; ++q)
      if (meet(out[o], out[q])) return DETFFN_ERR_INVALID_ARG;
  }
  return DETFFN_OK;
}

inline Span rows_span(const void* p, long long M, long long H, long long ld, long long es) {
  return Span{p, M, H * es, ld * es};
}
inline Span flat_span(const void* p, long long bytes) { return Span{p, 1, bytes, bytes}; }

inline detffn_status current_sms(int* sms) {
  int dev = 0;
  TRYCU(cudaGetDevice(&dev));
  return cu(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
}

}  // namespace detffn
