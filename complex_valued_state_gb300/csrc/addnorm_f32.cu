// The norm before a block, with the residual sum, for float32 tensors.

#include "addnorm_kernels.cuh"

namespace cssd {
namespace blocknorm {

cudaError_t add_f32(const AddNormArgs& a, cudaStream_t st) { return add_forward<float>(a, st); }
cudaError_t add_back_f32(const AddNormArgs& a, void* ws, cudaStream_t st) { return add_backward<float>(a, ws, st); }

}  // namespace blocknorm

}  // namespace cssd
