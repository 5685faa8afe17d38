// The backward of the norms around a block: float32 rows, without a norm behind the block.
#include "residual_norm_bwd.cuh"

namespace grpo {

cudaError_t resnorm_bwd_f32(const ResNormArgs& a, bool whole, int sms, int* walkers, cudaStream_t s) {
  return resnorm_bwd_kind<float, false>(a, whole, sms, walkers, s);
}

}  // namespace grpo
