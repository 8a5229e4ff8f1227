// The norms before and after a block, forward and gradients:
//   add    s = residual + alpha (scale x),  y = norm(s) w + b
//   gated  y = (norm(x) w + b) silu(z),  or  y = norm(x silu(z)) w + b  (the gate first), over groups of columns
// with norm(h) = (h - m) r, r = 1 / sqrt(mean((h - m)^2) + eps), m = mean(h) or (root mean square) 0.  With a
// the gradient of norm(h) and hh = norm(h),
//   dh = r (a - [mean(a)] - hh mean(a hh))        ([..]: where the mean is taken off)
// All are bound by the tensors' bytes.  Statistics and sums are fp32, the variance from the centred values; s is
// rounded to its type before the norm sees it, so that the gradients, which read s, are those of what was
// computed.  Sums over the rows are taken in a fixed order: a thread owns its columns over the rows of its CTA,
// and a second kernel adds up the CTAs' sums.

#include <type_traits>

#include "cssd_internal.h"
#include "delta_common.cuh"

namespace cssd {
namespace {

using delta::from_f;
using delta::to_f;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Sum over the TEAM threads that share a row (one warp, or a CTA of whole warps).
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* red, int tid) {
    v = warp_sum(v);
    if constexpr (TEAM > 32) {
        __syncthreads();
        if (tid % 32 == 0) red[tid / 32] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TEAM / 32; ++i) v += red[i];
    }
    return v;
}

template <typename W>
__device__ __forceinline__ float at_or(const W* w, int64_t i, float other) {
    return w ? to_f(w[i]) : other;
}
__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + __expf(-z)); }

// --------------------------------------------------------------- add, forward
template <typename E, typename R, typename W>
__global__ void __launch_bounds__(256) add_stream(AddNormArgs a) {
    __shared__ float red[8];
    const int tid = threadIdx.x;
    const float inv = 1.f / (float)a.width;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const E* x = static_cast<const E*>(a.x) + row * a.width;
        const R* res = static_cast<const R*>(a.residual) + row * a.width;
        const W *sc = static_cast<const W*>(a.scale), *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
        R* s = static_cast<R*>(a.s) + row * a.width;
        E* y = static_cast<E*>(a.y) + row * a.width;
        float t = 0.f;
        for (int64_t c = tid; c < a.width; c += 256) {
            s[c] = from_f<R>(fmaf(a.alpha, at_or(sc, c, 1.f) * to_f(x[c]), to_f(res[c])));
            t += to_f(s[c]);
        }
        const float m = a.layer ? team_sum<256>(t, red, tid) * inv : 0.f;
        t = 0.f;
        for (int64_t c = tid; c < a.width; c += 256) {
            const float d = to_f(s[c]) - m;
            t = fmaf(d, d, t);
        }
        const float r = rsqrtf(team_sum<256>(t, red, tid) * inv + a.eps);
        if (tid == 0) {
            if (a.mean && a.layer) a.mean[row] = m;
            if (a.rstd) a.rstd[row] = r;
        }
        for (int64_t c = tid; c < a.width; c += 256)
            y[c] = from_f<E>(fmaf((to_f(s[c]) - m) * r, at_or(w, c, 1.f), at_or(b, c, 0.f)));
    }
}

// --------------------------------------------------------------- gated, forward
template <typename E, typename W, int TEAM>
__global__ void __launch_bounds__(256) gated_stream(GatedNormArgs a) {
    __shared__ float red[8];
    const int tid = threadIdx.x % TEAM;
    const int64_t groups = a.width / a.group, units = a.rows * groups;
    const float inv = 1.f / (float)a.group;
    const W *w = static_cast<const W*>(a.weight), *b = static_cast<const W*>(a.bias);
    for (int64_t u = (int64_t)blockIdx.x * (256 / TEAM) + threadIdx.x / TEAM; u < units; u += (int64_t)gridDim.x * (256 / TEAM)) {
        const int64_t at = u * a.group, c0 = u % groups * a.group;
        const E *x = static_cast<const E*>(a.x) + at, *z = static_cast<const E*>(a.z) + at;
        E* y = static_cast<E*>(a.y) + at;
        auto h = [&](int64_t c) {
            const float xv = to_f(x[c]);
            if (!a.gate_first) return xv;
            const float zv = to_f(z[c]);
            return xv * (zv * sigmoid(zv));
        };
        float t = 0.f;
        if (a.layer)
            for (int64_t c = tid; c < a.group; c += TEAM) t += h(c);
        const float m = a.layer ? team_sum<TEAM>(t, red, tid) * inv : 0.f;
        t = 0.f;
        for (int64_t c = tid; c < a.group; c += TEAM) {
            const float d = h(c) - m;
            t = fmaf(d, d, t);
        }
        const float r = rsqrtf(team_sum<TEAM>(t, red, tid) * inv + a.eps);
        if (tid == 0) {
            if (a.mean && a.layer) a.mean[u] = m;
            if (a.rstd) a.rstd[u] = r;
        }
        for (int64_t c = tid; c < a.group; c += TEAM) {
            float v = fmaf((h(c) - m) * r, at_or(w, c0 + c, 1.f), at_or(b, c0 + c, 0.f));
            if (!a.gate_first) {
                const float zv = to_f(z[c]);
                v *= zv * sigmoid(zv);
            }
            y[c] = from_f<E>(v);
        }
    }
}

// --------------------------------------------------------------- gradients, streamed
// First the two means of every row (of every group), then dx and the column sums.
template <typename E, typename R, typename W>
__global__ void __launch_bounds__(256) add_back_sums(AddNormArgs a, float2* __restrict__ sums) {
    __shared__ float red[8];
    const W* w = static_cast<const W*>(a.weight);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const E* dy = static_cast<const E*>(a.dy) + row * a.width;
        const R* s = static_cast<const R*>(a.s) + row * a.width;
        const float m = a.layer ? a.mean[row] : 0.f, r = a.rstd[row];
        float s1 = 0.f, s2 = 0.f;
        for (int64_t c = threadIdx.x; c < a.width; c += 256) {
            const float g = to_f(dy[c]) * at_or(w, c, 1.f);
            s1 += g;
            s2 = fmaf(g, (to_f(s[c]) - m) * r, s2);
        }
        s1 = team_sum<256>(s1, red, threadIdx.x);
        s2 = team_sum<256>(s2, red, threadIdx.x);
        if (threadIdx.x == 0) sums[row] = make_float2(a.layer ? s1 / (float)a.width : 0.f, s2 / (float)a.width);
    }
}

// Column sums of a CTA of 32 columns x 8 row lanes, `which` of them, into part[blockIdx.y][which][width].
template <int K>
__device__ __forceinline__ void put_columns(const float (&v)[K], float (&red)[K][8][33], float* part, int64_t c, int64_t width) {
    const int lx = threadIdx.x % 32, ly = threadIdx.x / 32;
#pragma unroll
    for (int e = 0; e < K; ++e) red[e][ly][lx] = v[e];
    __syncthreads();
    if (ly < K && c < width) {
        float s = 0.f;
        for (int i = 0; i < 8; ++i) s += red[ly][i][lx];
        part[((int64_t)blockIdx.y * K + ly) * width + c] = s;
    }
}

template <typename E, typename R, typename W>
__global__ void __launch_bounds__(256) add_back_cols(AddNormArgs a, const float2* __restrict__ sums, float* __restrict__ part) {
    __shared__ float red[3][8][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32, width = a.width;
    float sum[3] = {};  // of scale, weight, bias
    if (c < width) {
        const E *x = static_cast<const E*>(a.x), *dy = static_cast<const E*>(a.dy);
        const R *s = static_cast<const R*>(a.s), *ds = static_cast<const R*>(a.ds);
        const float wv = at_or(static_cast<const W*>(a.weight), c, 1.f), sv = a.alpha * at_or(static_cast<const W*>(a.scale), c, 1.f);
        for (int64_t row = (int64_t)blockIdx.y * 8 + threadIdx.x / 32; row < a.rows; row += (int64_t)gridDim.y * 8) {
            const int64_t i = row * width + c;
            const float m = a.layer ? a.mean[row] : 0.f, r = a.rstd[row], d = to_f(dy[i]), hh = (to_f(s[i]) - m) * r;
            const float2 u = sums[row];
            const float t = fmaf(r, d * wv - u.x - hh * u.y, ds ? to_f(ds[i]) : 0.f);
            if (a.gscale) sum[0] = fmaf(t, to_f(x[i]), sum[0]);
            sum[1] = fmaf(d, hh, sum[1]);
            sum[2] += d;
            static_cast<R*>(a.gresidual)[i] = from_f<R>(t);
            static_cast<E*>(a.gx)[i] = from_f<E>(sv * t);
        }
        sum[0] *= a.alpha;
    }
    put_columns(sum, red, part, c, width);
}

// What a column needs of the gate: silu and its slope.
__device__ __forceinline__ void gate_of(float z, float& gate, float& slope) {
    const float s = sigmoid(z);
    gate = z * s;
    slope = s * fmaf(z, 1.f - s, 1.f);
}

template <typename E, typename W, int TEAM>
__global__ void __launch_bounds__(256) gated_back_sums(GatedNormArgs a, float2* __restrict__ sums) {
    __shared__ float red[8];
    const int tid = threadIdx.x % TEAM;
    const int64_t groups = a.width / a.group, units = a.rows * groups;
    const W* w = static_cast<const W*>(a.weight);
    for (int64_t u = (int64_t)blockIdx.x * (256 / TEAM) + threadIdx.x / TEAM; u < units; u += (int64_t)gridDim.x * (256 / TEAM)) {
        const int64_t at = u * a.group, c0 = u % groups * a.group;
        const float m = a.layer ? a.mean[u] : 0.f, r = a.rstd[u];
        float s1 = 0.f, s2 = 0.f;
        for (int64_t c = tid; c < a.group; c += TEAM) {
            float gate, slope, xv = to_f(static_cast<const E*>(a.x)[at + c]), d = to_f(static_cast<const E*>(a.dy)[at + c]);
            gate_of(to_f(static_cast<const E*>(a.z)[at + c]), gate, slope);
            (a.gate_first ? xv : d) *= gate;
            const float g = d * at_or(w, c0 + c, 1.f);
            s1 += g;
            s2 = fmaf(g, (xv - m) * r, s2);
        }
        s1 = team_sum<TEAM>(s1, red, tid);
        s2 = team_sum<TEAM>(s2, red, tid);
        if (tid == 0) sums[u] = make_float2(a.layer ? s1 / (float)a.group : 0.f, s2 / (float)a.group);
    }
}

template <typename E, typename W>
__global__ void __launch_bounds__(256) gated_back_cols(GatedNormArgs a, const float2* __restrict__ sums, float* __restrict__ part) {
    __shared__ float red[2][8][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32, width = a.width, groups = width / a.group;
    float sum[2] = {};
    if (c < width) {
        const E *x = static_cast<const E*>(a.x), *z = static_cast<const E*>(a.z), *dy = static_cast<const E*>(a.dy);
        const float wv = at_or(static_cast<const W*>(a.weight), c, 1.f), bv = at_or(static_cast<const W*>(a.bias), c, 0.f);
        const int64_t gi = c / a.group;
        for (int64_t row = (int64_t)blockIdx.y * 8 + threadIdx.x / 32; row < a.rows; row += (int64_t)gridDim.y * 8) {
            const int64_t i = row * width + c, u = row * groups + gi;
            const float m = a.layer ? a.mean[u] : 0.f, r = a.rstd[u], xv = to_f(x[i]), d = to_f(dy[i]);
            float gate, slope;
            gate_of(to_f(z[i]), gate, slope);
            const float hh = ((a.gate_first ? xv * gate : xv) - m) * r, du = a.gate_first ? d : d * gate;
            const float2 t = sums[u];
            const float dh = r * (du * wv - t.x - hh * t.y);
            sum[0] = fmaf(du, hh, sum[0]);
            sum[1] += du;
            static_cast<E*>(a.gx)[i] = from_f<E>(a.gate_first ? dh * gate : dh);
            static_cast<E*>(a.gz)[i] = from_f<E>((a.gate_first ? dh * xv : d * fmaf(hh, wv, bv)) * slope);
        }
    }
    put_columns(sum, red, part, c, width);
}

// part [n][k][width] -> the k vectors (null: not wanted): 32 columns x 32 lanes over n, in a fixed order.
template <typename W>
struct Vectors {
    W* to[3];
};
template <typename W>
__global__ void __launch_bounds__(1024) join_columns(const float* part, int n, int64_t width, Vectors<W> out) {
    __shared__ float red[32][33];
    W* to = out.to[blockIdx.y];
    if (!to) return;
    const int lx = threadIdx.x % 32, ly = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lx;
    float s = 0.f;
    delta::wait_for_previous();  // (nothing of `part` is read before)
    if (c < width)
#pragma unroll 8
        for (int i = ly; i < n; i += 32) s += part[((int64_t)i * gridDim.y + blockIdx.y) * width + c];
    red[ly][lx] = s;
    __syncthreads();
    s = warp_sum(red[lx][ly]);  // column ly, over the lanes
    const int64_t oc = (int64_t)blockIdx.x * 32 + ly;
    if (lx == 0 && oc < width) to[oc] = from_f<W>(s);
}

constexpr int kBackGrid = 304;  // CTAs of the gradients along the rows: two an SM (152 SMs)
int back_groups(int64_t rows) { return (int)(rows < kBackGrid ? rows : kBackGrid); }
unsigned grid_of(int64_t units, int64_t most) { return (unsigned)(units < most ? units : most); }

template <typename W>
cudaError_t join(const float* part, int n, int64_t width, int k, W* a, W* b, W* c, cudaStream_t st) {
    if (!a && !b && !c) return cudaSuccess;
    // launched while the kernel before it runs, so that its CTAs are there when that ends
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((width + 31) / 32), k);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_columns<W>, part, n, width, Vectors<W>{{a, b, c}});
}

template <typename E, typename R, typename W>
cudaError_t add_fwd(const AddNormArgs& a, cudaStream_t st) {
    add_stream<E, R, W><<<grid_of(a.rows, 8192), 256, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename E, typename R, typename W>
cudaError_t add_bwd(const AddNormArgs& a, void* ws, cudaStream_t st) {
    float2* sums = static_cast<float2*>(ws);
    float* part = reinterpret_cast<float*>(sums + a.rows);
    const int n = back_groups(a.rows);
    add_back_sums<E, R, W><<<grid_of(a.rows, 8192), 256, 0, st>>>(a, sums);
    add_back_cols<E, R, W><<<dim3((unsigned)((a.width + 31) / 32), n), 256, 0, st>>>(a, sums, part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return join<W>(part, n, a.width, 3, static_cast<W*>(a.gscale), static_cast<W*>(a.gweight), static_cast<W*>(a.gbias), st);
}

template <typename E, typename W>
cudaError_t gated_fwd(const GatedNormArgs& a, cudaStream_t st) {
    const int64_t units = a.rows * (a.width / a.group);
    if (a.group <= 1024)
        gated_stream<E, W, 32><<<grid_of((units + 7) / 8, 8192), 256, 0, st>>>(a);
    else
        gated_stream<E, W, 256><<<grid_of(units, 8192), 256, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename E, typename W>
cudaError_t gated_bwd(const GatedNormArgs& a, void* ws, cudaStream_t st) {
    const int64_t units = a.rows * (a.width / a.group);
    float2* sums = static_cast<float2*>(ws);
    float* part = reinterpret_cast<float*>(sums + units);
    const int n = back_groups(a.rows);
    if (a.group <= 1024)
        gated_back_sums<E, W, 32><<<grid_of((units + 7) / 8, 8192), 256, 0, st>>>(a, sums);
    else
        gated_back_sums<E, W, 256><<<grid_of(units, 8192), 256, 0, st>>>(a, sums);
    gated_back_cols<E, W><<<dim3((unsigned)((a.width + 31) / 32), n), 256, 0, st>>>(a, sums, part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return join<W>(part, n, a.width, 2, static_cast<W*>(a.gweight), static_cast<W*>(a.gbias), static_cast<W*>(nullptr), st);
}

// Calls f with null pointers of the tensors' type and of another that is either it or float.
template <typename F>
cudaError_t by_types(int xtype, F f) {
    if (xtype == CSSD_BF16) return f(static_cast<__nv_bfloat16*>(nullptr));
    if (xtype == CSSD_F16) return f(static_cast<__half*>(nullptr));
    return f(static_cast<float*>(nullptr));
}
template <typename E, typename F>
cudaError_t or_float(bool wide, E* e, F f) {
    if constexpr (!std::is_same_v<E, float>)
        if (!wide) return f(e);
    return f(static_cast<float*>(nullptr));
}
template <typename F>
cudaError_t add_types(const AddNormArgs& a, F f) {
    return by_types(a.xtype, [&](auto* e) {
        return or_float(a.rtype == CSSD_F32, e, [&](auto* r) {
            return or_float(a.wtype == CSSD_F32, e, [&](auto* w) { return f(e, r, w); });
        });
    });
}
template <typename F>
cudaError_t gated_types(const GatedNormArgs& a, F f) {
    return by_types(a.xtype, [&](auto* e) { return or_float(a.wtype == CSSD_F32, e, [&](auto* w) { return f(e, w); }); });
}
template <typename P>
using To = std::remove_pointer_t<P>;

}  // namespace

size_t add_norm_backward_workspace_bytes(int64_t rows, int64_t width) {
    return sizeof(float) * (2 * (size_t)rows + (size_t)back_groups(rows) * 3 * (size_t)width);
}
cudaError_t launch_add_norm(const AddNormArgs& a, cudaStream_t st) {
    return add_types(a, [&](auto* e, auto* r, auto* w) { return add_fwd<To<decltype(e)>, To<decltype(r)>, To<decltype(w)>>(a, st); });
}
cudaError_t launch_add_norm_backward(const AddNormArgs& a, void* ws, cudaStream_t st) {
    return add_types(a, [&](auto* e, auto* r, auto* w) { return add_bwd<To<decltype(e)>, To<decltype(r)>, To<decltype(w)>>(a, ws, st); });
}

size_t gated_norm_backward_workspace_bytes(int64_t rows, int64_t width, int64_t group) {
    return sizeof(float) * (2 * (size_t)rows * (size_t)(width / group) + (size_t)back_groups(rows) * 2 * (size_t)width);
}
cudaError_t launch_gated_norm(const GatedNormArgs& a, cudaStream_t st) {
    return gated_types(a, [&](auto* e, auto* w) { return gated_fwd<To<decltype(e)>, To<decltype(w)>>(a, st); });
}
cudaError_t launch_gated_norm_backward(const GatedNormArgs& a, void* ws, cudaStream_t st) {
    return gated_types(a, [&](auto* e, auto* w) { return gated_bwd<To<decltype(e)>, To<decltype(w)>>(a, ws, st); });
}

}  // namespace cssd
