// Layer norm backward of one storage format.
#include "rr_norm.cuh"

namespace rr {
cudaError_t launch_norm_grad_f16(const NormGradParams &p, cudaStream_t s) {
  return p.wtype == kF32 ? norm::backward<kF16, kF32>(p, s) : norm::backward<kF16, kF16>(p, s);
}
}  // namespace rr
