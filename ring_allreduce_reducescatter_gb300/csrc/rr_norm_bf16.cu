// Layer norm forward of one storage format.
#include "rr_norm.cuh"

namespace rr {
cudaError_t launch_norm_bf16(const NormParams &p, cudaStream_t s) {
  return p.wtype == kF32 ? norm::forward<kBF16, kF32>(p, s) : norm::forward<kBF16, kBF16>(p, s);
}
}  // namespace rr
