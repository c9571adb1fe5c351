// k_join_bf16.cu -- the residual join's kernels for BF16 elements.
#include "k_join_ring.cuh"

namespace detffn {
cudaError_t join_forward_bf16(const JoinArgs& a, cudaStream_t st) { return join::forward<DETFFN_BF16>(a, st); }
cudaError_t join_backward_bf16(const JoinArgs& a, cudaStream_t st) { return join::backward<DETFFN_BF16>(a, st); }
}  // namespace detffn
