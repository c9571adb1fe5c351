// k_join_f16.cu -- the residual join's kernels for F16 elements.
#include "k_join_ring.cuh"

namespace detffn {
cudaError_t join_forward_f16(const JoinArgs& a, cudaStream_t st) { return join::forward<DETFFN_F16>(a, st); }
cudaError_t join_backward_f16(const JoinArgs& a, cudaStream_t st) { return join::backward<DETFFN_F16>(a, st); }
}  // namespace detffn
