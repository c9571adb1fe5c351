// moe.h -- launchers of the mixture-of-experts layer for a few tokens.
#pragma once

#include "common.cuh"

namespace detffn {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;
constexpr long long kMoeMaxWidth = 65536;  // of H and I

struct MoeArgs {
  const void *x = nullptr, *Wr = nullptr, *Wg = nullptr, *Wu = nullptr, *Wd = nullptr;
  void* out = nullptr;
  int T = 0, E = 0, k = 0, dtype = 0, normalize = 0;
  long long H = 0, I = 0;
  // Results of the routing: experts and weights [T][k], slot 0 the largest.
  int* experts = nullptr;
  float* weights = nullptr;
  // Workspace: logits [T][E]; pos [T][k], the place of a token's slot among
  // the pairs ordered by expert; pair [T * k], the token * k + slot at each
  // place; first [E + 1], each expert's first place; h [T * k][I].
  float* logits = nullptr;
  int *pos = nullptr, *pair = nullptr, *first = nullptr;
  void* h = nullptr;
};

// CUDA-core kernels for any sizes (FP32, FP16 or BF16).
cudaError_t launch_moe_general(const MoeArgs& a, cudaStream_t st);

}  // namespace detffn
