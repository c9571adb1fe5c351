// grouped.h -- launchers of matrix products grouped by expert.
#pragma once

#include "block.h"

namespace detffn {

constexpr int kGroupedMaxExperts = 1024;
constexpr long long kGroupedMaxWidth = 65536;        // of K and N
constexpr long long kGroupedMaxRows = (1ll << 31) - 256;   // (a count of rows and a tile of 256 add up in an int)

// Expert e has rows [off[e], off[e + 1]) of x [R, K] and of out, dOut [R, N],
// and the matrix W[e] [N, K].
struct GroupedArgs {
  long long R = 0, K = 0, N = 0;
  int E = 0, dtype = 0;
  const int* off = nullptr;
  Rows x, out;                     // forward: out[r] = W[e] x[r]
  const void* W = nullptr;         // [E * N][K], rows ldw apart (the CUDA-core kernels: K)
  long long ldw = 0;
  Rows dout, dx;                   // backward: dx[r] = W[e]^T dout[r]
  void* dW = nullptr;              //   dW[e] = sum over the expert's rows of dout[r] x[r]^T
};

enum class Grouped { kForward, kInput, kWeight };   // out, dx, dW

// Whether rows of a 16-bit type lie on 16-byte boundaries, as the tensor kernel's
// loads need them.
inline bool grouped_boundary(const Rows& r, long long rows) {
  return (uintptr_t)r.p % 16 == 0 && (rows <= 1 || r.ld % 8 == 0);
}
constexpr long long grouped_pad(long long n) { return (n + 7) / 8 * 8; }
// to[r * grouped_pad(width) + c] = from's element (r, c), 16-bit types.
cudaError_t launch_grouped_rows(const Rows& from, long long rows, long long width, uint16_t* to, int sm_count, cudaStream_t st);
// The same of a.W; matrices of experts without rows may be left out.
cudaError_t launch_grouped_matrices(const GroupedArgs& a, uint16_t* to, int sm_count, cudaStream_t st);

// Tensor-core kernel: BF16 and FP16, rows of x, W and dout (those it reads) on
// 16-byte boundaries.
cudaError_t launch_grouped_tensor(const GroupedArgs& a, Grouped what, const Waits& wt, int sm_count, cudaStream_t st);

// CUDA-core kernels for any sizes, strides and types.
cudaError_t launch_grouped_general(const GroupedArgs& a, Grouped what, int sm_count, cudaStream_t st);

}  // namespace detffn
