// Linear attention with a decay for each head: the kernels for float32 tensors.

#include "linattn_kernels.cuh"

namespace cssd {
namespace linattn {

cudaError_t forward_f32(const LinattnArgs& a, void* ws, cudaStream_t st) { return forward_of<float>(a, ws, st); }
cudaError_t backward_f32(const LinattnArgs& a, void* ws, cudaStream_t st) { return backward_of<float>(a, ws, st); }

}  // namespace linattn

}  // namespace cssd
