// Layer norm forward of one storage format.
#include "rr_norm.cuh"

namespace rr {
cudaError_t launch_norm_f16(const NormParams &p, cudaStream_t s) {
  return p.wtype == kF32 ? norm::forward<kF16, kF32>(p, s) : norm::forward<kF16, kF16>(p, s);
}
}  // namespace rr
