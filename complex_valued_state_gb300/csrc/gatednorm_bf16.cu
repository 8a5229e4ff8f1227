// The gated norm after a mixer for bfloat16 tensors.

#include "gatednorm_kernels.cuh"

namespace cssd {
namespace blocknorm {

cudaError_t gated_bf16(const GatedNormArgs& a, cudaStream_t st) { return gated_forward<__nv_bfloat16>(a, st); }
cudaError_t gated_back_bf16(const GatedNormArgs& a, void* ws, cudaStream_t st) { return gated_backward<__nv_bfloat16>(a, ws, st); }

}  // namespace blocknorm

size_t gated_norm_backward_workspace_bytes(int64_t rows, int64_t width, int64_t group) {
    return sizeof(float) * (2 * (size_t)rows * (size_t)(width / group) + (size_t)back_groups(rows) * 2 * (size_t)width);
}
cudaError_t launch_gated_norm(const GatedNormArgs& a, cudaStream_t st) {
    if (a.xtype == CSSD_BF16) return blocknorm::gated_bf16(a, st);
    if (a.xtype == CSSD_F16) return blocknorm::gated_f16(a, st);
    return blocknorm::gated_f32(a, st);
}
cudaError_t launch_gated_norm_backward(const GatedNormArgs& a, void* ws, cudaStream_t st) {
    if (a.xtype == CSSD_BF16) return blocknorm::gated_back_bf16(a, ws, st);
    if (a.xtype == CSSD_F16) return blocknorm::gated_back_f16(a, ws, st);
    return blocknorm::gated_back_f32(a, ws, st);
}

}  // namespace cssd
