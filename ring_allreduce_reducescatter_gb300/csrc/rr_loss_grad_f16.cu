// The linear cross entropy's gradient of one storage format.
#include "rr_loss_grad.cuh"

namespace rr {
cudaError_t launch_loss_grad_f16(const LossGradParams &p, cudaStream_t s) { return loss::backward<kF16>(p, s); }
}  // namespace rr
