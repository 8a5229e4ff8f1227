// The gated norm after a mixer for float16 tensors.

#include "gatednorm_kernels.cuh"

namespace cssd {
namespace blocknorm {

cudaError_t gated_f16(const GatedNormArgs& a, cudaStream_t st) { return gated_forward<__half>(a, st); }
cudaError_t gated_back_f16(const GatedNormArgs& a, void* ws, cudaStream_t st) { return gated_backward<__half>(a, ws, st); }

}  // namespace blocknorm

}  // namespace cssd
