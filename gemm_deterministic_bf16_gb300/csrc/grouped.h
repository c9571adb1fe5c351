// grouped.h -- launchers of matrix products grouped by expert.
#pragma once

#include "block.h"

namespace detffn {

constexpr int kGroupedMaxExperts = 1024;
constexpr long long kGroupedMaxWidth = 65536;        // of K and N
constexpr long long kGroupedMaxRows = (1ll << 31) - 1;

// Expert e has rows [off[e], off[e + 1]) of x [R, K] and of out, dOut [R, N],
// and the matrix W[e] [N, K].
struct GroupedArgs {
  long long R = 0, K = 0, N = 0;
  int E = 0, dtype = 0;
  const int* off = nullptr;
  Rows x, out;                     // forward: out[r] = W[e] x[r]
  const void* W = nullptr;
  Rows dout, dx;                   // backward: dx[r] = W[e]^T dout[r]
  void* dW = nullptr;              //   dW[e] = sum over the expert's rows of dout[r] x[r]^T
};

enum class Grouped { kForward, kInput, kWeight };   // out, dx, dW

// Tensor-core kernel: BF16 and FP16, K and N multiples of 8, x, W and dout on
// 16-byte boundaries.
bool grouped_tensor_covers(const GroupedArgs& a, Grouped what);
cudaError_t launch_grouped_tensor(const GroupedArgs& a, Grouped what, const Waits& wt, int sm_count, cudaStream_t st);

// CUDA-core kernels for any sizes, strides and types.
cudaError_t launch_grouped_general(const GroupedArgs& a, Grouped what, int sm_count, cudaStream_t st);

}  // namespace detffn
