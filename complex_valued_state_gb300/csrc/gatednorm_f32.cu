// The gated norm after a mixer for float32 tensors.

#include "gatednorm_kernels.cuh"

namespace cssd {
namespace blocknorm {

cudaError_t gated_f32(const GatedNormArgs& a, cudaStream_t st) { return gated_forward<float>(a, st); }
cudaError_t gated_back_f32(const GatedNormArgs& a, void* ws, cudaStream_t st) { return gated_backward<float>(a, ws, st); }

}  // namespace blocknorm

}  // namespace cssd
