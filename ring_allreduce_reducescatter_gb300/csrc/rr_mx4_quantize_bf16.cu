// rr_mx4_quantize_bf16.cu -- the quantisation kernels of one storage format.
#include "rr_mx4_quantize.cuh"

namespace rr {

cudaError_t launch_mx4_quantize_bf16(const QuantParams &p, cudaStream_t s) { return mx4q::quantize_any<kBF16>(p, s); }

}  // namespace rr
