// Linear attention with a decay for each head: the kernels for bfloat16 tensors.

#include "linattn_kernels.cuh"

namespace cssd {
namespace linattn {

cudaError_t forward_bf16(const LinattnArgs& a, void* ws, cudaStream_t st) { return forward_of<__nv_bfloat16>(a, ws, st); }
cudaError_t backward_bf16(const LinattnArgs& a, void* ws, cudaStream_t st) { return backward_of<__nv_bfloat16>(a, ws, st); }

size_t forward_bytes(const LinattnArgs& a) { return scratch_bytes(a, 1); }
size_t backward_bytes(const LinattnArgs& a) {
    const size_t chunks = (size_t)a.Bz * a.H * shape_of(a, 2).nc;
    return scratch_bytes(a, 2) + parts_bytes(a) + up(chunks * 4);
}

}  // namespace linattn

size_t linattn_workspace_bytes(const LinattnArgs& a) { return linattn::forward_bytes(a); }
size_t linattn_backward_workspace_bytes(const LinattnArgs& a) { return linattn::backward_bytes(a); }

cudaError_t launch_linattn_forward(const LinattnArgs& a, void* ws, cudaStream_t st) {
    if (a.dtype == CSSD_BF16) return linattn::forward_bf16(a, ws, st);
    if (a.dtype == CSSD_F16) return linattn::forward_f16(a, ws, st);
    return linattn::forward_f32(a, ws, st);
}
cudaError_t launch_linattn_backward(const LinattnArgs& a, void* ws, cudaStream_t st) {
    if (a.dtype == CSSD_BF16) return linattn::backward_bf16(a, ws, st);
    if (a.dtype == CSSD_F16) return linattn::backward_f16(a, ws, st);
    return linattn::backward_f32(a, ws, st);
}

}  // namespace cssd
