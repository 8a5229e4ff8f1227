// The norm before a block, with the residual sum, for float16 tensors.

#include "addnorm_kernels.cuh"

namespace cssd {
namespace blocknorm {

cudaError_t add_f16(const AddNormArgs& a, cudaStream_t st) { return add_forward<__half>(a, st); }
cudaError_t add_back_f16(const AddNormArgs& a, void* ws, cudaStream_t st) { return add_backward<__half>(a, ws, st); }

}  // namespace blocknorm

}  // namespace cssd
