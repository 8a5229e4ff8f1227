// The norm before a block, with the residual sum, for bfloat16 tensors.

#include "addnorm_kernels.cuh"

namespace cssd {
namespace blocknorm {

cudaError_t add_bf16(const AddNormArgs& a, cudaStream_t st) { return add_forward<__nv_bfloat16>(a, st); }
cudaError_t add_back_bf16(const AddNormArgs& a, void* ws, cudaStream_t st) { return add_backward<__nv_bfloat16>(a, ws, st); }

}  // namespace blocknorm

size_t add_norm_backward_workspace_bytes(int64_t rows, int64_t width) {
    return sizeof(float) * (2 * (size_t)rows + (size_t)back_groups(rows) * 3 * (size_t)width);
}
cudaError_t launch_add_norm(const AddNormArgs& a, cudaStream_t st) {
    if (a.xtype == CSSD_BF16) return blocknorm::add_bf16(a, st);
    if (a.xtype == CSSD_F16) return blocknorm::add_f16(a, st);
    return blocknorm::add_f32(a, st);
}
cudaError_t launch_add_norm_backward(const AddNormArgs& a, void* ws, cudaStream_t st) {
    if (a.xtype == CSSD_BF16) return blocknorm::add_back_bf16(a, ws, st);
    if (a.xtype == CSSD_F16) return blocknorm::add_back_f16(a, ws, st);
    return blocknorm::add_back_f32(a, ws, st);
}

}  // namespace cssd
