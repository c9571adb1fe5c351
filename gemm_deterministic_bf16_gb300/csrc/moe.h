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
  // place; first [E + 1], each expert's first place; h, FP32
  // [T * k][I] or two terms [2][T * k][I] of the stored type.
  float* logits = nullptr;
  int *pos = nullptr, *pair = nullptr, *first = nullptr;
  void* h = nullptr;
};

// More workspace: the tensor kernel's counters [1 + E + ceil(H / 128) + T * k],
// the pairs' outputs y [parts][T * k][H] in FP32 (the general kernels use one
// part), and for FP16 the tensor kernel's h in FP32, [T * k][I].
struct MoeScratch {
  int* counters = nullptr;
  float* y = nullptr;
  float* h32 = nullptr;
};

// Router logits; block 0 clears n counters.
cudaError_t launch_moe_logits(const MoeArgs& a, int* counters, int n, cudaStream_t st);

// The parts a down projection's K is summed in, and the 128-wide stages of a part.
void moe_parts(long long H, long long I, int* parts, int* stages);

// Tensor-core kernels (BF16 and FP16, widths multiples of 8, 16-byte-aligned
// tensors).
bool moe_tensor_covers(const MoeArgs& a);
cudaError_t launch_moe_tensor(const MoeArgs& a, const MoeScratch& sc, const Waits& wt, int sm_count, cudaStream_t st);

// CUDA-core kernels for any sizes (FP32, FP16 or BF16).
cudaError_t launch_moe_general(const MoeArgs& a, const MoeScratch& sc, cudaStream_t st);

}  // namespace detffn
