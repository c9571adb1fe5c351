// w4.h -- launchers of the products with 4-bit weights.
#pragma once

#include "common.cuh"

namespace detffn {

constexpr int kW4Run = 128;                  // codes of a row that are laid out together, 64 bytes
constexpr long long kW4MaxWidth = 1 << 20;   // of K and N
constexpr int kW4MaxTokens = 64;

// N rows of K codes (64 bytes a run) with one scale for `group` codes of a row.
struct W4Matrix {
  const uint8_t* codes = nullptr;
  const void* scales = nullptr;   // [N][ceil(K / group)], stype
  long long N = 0, K = 0;
  int group = 0, stype = 0;
};

// Activations as the kernels read them: 16-bit values (BF16 or FP16) on 16-byte
// boundaries, row strides a multiple of 8.  An FP32 activation is the sum of
// `terms` BF16 values, `plane` elements apart.
struct W4Rows {
  const void* p = nullptr;
  long long ld = 0, plane = 0;
  int terms = 1;
  bool f16 = false;
};
constexpr long long w4_pad(long long n) { return (n + 7) / 8 * 8; }
// Whether rows of a 16-bit type can be read where they are.
inline bool w4_in_place(const void* p, long long ld, long long T, long long K) {
  return (uintptr_t)p % 16 == 0 && K % 8 == 0 && (T <= 1 || ld % 8 == 0);
}

// out[t * ldo + n] in otype; with w2 = up's matrix (w gate's), SiLU(gate) up as
// `terms` planes of BF16.
struct W4Args {
  W4Matrix w, w2;
  W4Rows x;
  int T = 0;
  void* out = nullptr;
  long long ldo = 0, plane = 0;
  int otype = 0, terms = 1;
};

// x [T, K] of a type as W4Rows at `to` (terms planes of [T][w4_pad(K)]).
cudaError_t launch_w4_rows(const void* x, long long ldx, int dtype, long long T, long long K, int terms, void* to,
                           int sm_count, cudaStream_t st);
cudaError_t launch_w4_matvec(const W4Args& a, int sm_count, cudaStream_t st);
cudaError_t launch_w4_pack(const void* w, long long ld, int dtype, const W4Matrix& to, int sm_count, cudaStream_t st);
cudaError_t launch_w4_unpack(const W4Matrix& from, void* w, long long ld, int dtype, int sm_count, cudaStream_t st);

}  // namespace detffn
