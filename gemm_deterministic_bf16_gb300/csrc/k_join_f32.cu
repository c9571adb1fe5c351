// k_join_f32.cu -- the residual join's kernels for F32 elements.
#include "k_join_ring.cuh"

namespace detffn {
cudaError_t join_forward_f32(const JoinArgs& a, cudaStream_t st) { return join::forward<DETFFN_F32>(a, st); }
cudaError_t join_backward_f32(const JoinArgs& a, cudaStream_t st) { return join::backward<DETFFN_F32>(a, st); }
}  // namespace detffn
