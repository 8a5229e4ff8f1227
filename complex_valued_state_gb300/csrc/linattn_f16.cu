// Linear attention with a decay for each head: the kernels for float16 tensors.

#include "linattn_kernels.cuh"

namespace cssd {
namespace linattn {

cudaError_t forward_f16(const LinattnArgs& a, void* ws, cudaStream_t st) { return forward_of<__half>(a, ws, st); }
cudaError_t backward_f16(const LinattnArgs& a, void* ws, cudaStream_t st) { return backward_of<__half>(a, ws, st); }

}  // namespace linattn

}  // namespace cssd
