// Layer norm backward of one storage format.
#include "rr_norm.cuh"

namespace rr {
cudaError_t launch_norm_grad_bf16(const NormGradParams &p, cudaStream_t s) {
  return p.wtype == kF32 ? norm::backward<kBF16, kF32>(p, s) : norm::backward<kBF16, kBF16>(p, s);
}
}  // namespace rr
