// rr_mx4_quantize_f16.cu -- the quantisation kernels of one storage format.
#include "rr_mx4_quantize.cuh"

namespace rr {

cudaError_t launch_mx4_quantize_f16(const QuantParams &p, cudaStream_t s) { return mx4q::quantize_any<kF16>(p, s); }

}  // namespace rr
