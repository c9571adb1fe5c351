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

// out[t * N + n] (xtype, or FP32 where out32) of x[t * ldx + k] (xtype).
struct W4Args {
  W4Matrix w, w2;                 // w2.codes: gate w and up w2, out = SiLU(gate) up
  const void* x = nullptr;
  long long ldx = 0;
  void* out = nullptr;
  long long ldo = 0;
  int T = 0;
  int xtype = 0;
  int otype = 0;
  int terms = 0;                  // of an FP32 x: 3 (all 24 bits) or 2 (16 bits)
};

cudaError_t launch_w4_matvec(const W4Args& a, int sm_count, cudaStream_t st);
cudaError_t launch_w4_pack(const void* w, long long ld, int dtype, const W4Matrix& to, int sm_count, cudaStream_t st);
cudaError_t launch_w4_unpack(const W4Matrix& from, void* w, long long ld, int dtype, int sm_count, cudaStream_t st);

}  // namespace detffn
