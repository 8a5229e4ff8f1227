// Layer norm over the last axis, forward and gradients:
//     y  = (x - m) r w + b,  m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps)
//     a  = dy w,  xh = (x - m) r
//     dx = r (a - mean(a) - xh mean(a xh)),  dw = sum_rows dy xh,  db = sum_rows dy
// Both are bound by the tensors' bytes (x once and y once; x, dy once and dx
// once).  Statistics and sums are fp32, the variance from the centred values.
//
// Widths whose rows are whole 16-byte vectors and fit the threads' registers
// are read once and kept there; the others (odd widths, very wide rows) take
// the streaming kernels, which read a row again from the caches for each
// sum.  dw and db are summed in a fixed order: a thread owns its columns over
// the rows of its CTA, and the CTAs' sums are added up by a second kernel.

#include <type_traits>

#include <type_traits>

#include "cssd_internal.h"
#include "delta_common.cuh"

namespace cssd {
namespace {

using delta::from_f;
using delta::to_f;

constexpr int kMaxWarps = 32;

template <typename E>
struct Vec {
    static constexpr int W = 16 / sizeof(E);
};

template <typename E>
__device__ __forceinline__ void unpack(const uint4& raw, float (&f)[Vec<E>::W]) {
    alignas(16) E t[Vec<E>::W];
    *reinterpret_cast<uint4*>(t) = raw;
#pragma unroll
    for (int i = 0; i < Vec<E>::W; ++i) f[i] = to_f(t[i]);
}
template <typename E>
__device__ __forceinline__ uint4 pack(const float (&f)[Vec<E>::W]) {
    alignas(16) E t[Vec<E>::W];
#pragma unroll
    for (int i = 0; i < Vec<E>::W; ++i) t[i] = from_f<E>(f[i]);
    return *reinterpret_cast<uint4*>(t);
}
// W consecutive weights (16-byte aligned when the row is).
template <typename WT, int W>
__device__ __forceinline__ void load_w(const WT* w, int64_t at, float other, float (&f)[W]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] = other;
        return;
    }
    alignas(16) WT t[W];
    static_assert(sizeof(t) % 16 == 0, "whole vectors");
#pragma unroll
    for (int i = 0; i < (int)(sizeof(t) / 16); ++i)
        reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(w + at)[i];
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = to_f(t[i]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Sum over a row's TPR threads (whole warps of one CTA, or one warp).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red, int tid) {
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        __syncthreads();
        if (tid % 32 == 0) red[tid / 32] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v += red[i];
    }
    return v;
}

// --------------------------------------------------------------- forward
// TPR threads a row, the row in registers as IT vectors a thread; with one
// warp a row, RPC rows a CTA and no barrier.
template <typename E, typename WT, int TPR, int IT>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) norm_rows(const E* x, const WT* __restrict__ w,
                                                                  const WT* __restrict__ bias, float eps,
                                                                  E* y, float* __restrict__ mean,
                                                                  float* __restrict__ rstd, int64_t rows, int width) {
    constexpr int W = Vec<E>::W, RPC = TPR == 32 ? 4 : 1;
    __shared__ float red[kMaxWarps];
    const int tid = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPC + threadIdx.x / TPR;
    if (row >= rows) return;  // (whole warps; with barriers a CTA has one row)
    const int nv = width / W;
    const uint4* xr = reinterpret_cast<const uint4*>(x + row * width);
    uint4 raw[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = tid + TPR * i;
        raw[i] = c < nv ? __ldcs(xr + c) : make_uint4(0, 0, 0, 0);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        float f[W];
        unpack<E>(raw[i], f);
#pragma unroll
        for (int u = 0; u < W; ++u) sum += f[u];
    }
    const float inv = 1.f / (float)width;
    const float m = row_sum<TPR>(sum, red, tid) * inv;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        float f[W];
        unpack<E>(raw[i], f);
        if (tid + TPR * i < nv)
#pragma unroll
            for (int u = 0; u < W; ++u) sq = fmaf(f[u] - m, f[u] - m, sq);
    }
    const float r = rsqrtf(row_sum<TPR>(sq, red, tid) * inv + eps);
    if (tid == 0) {
        if (mean) mean[row] = m;
        if (rstd) rstd[row] = r;
    }
    uint4* yr = reinterpret_cast<uint4*>(y + row * width);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = tid + TPR * i;
        if (c >= nv) break;
        float f[W], wv[W], bv[W];
        unpack<E>(raw[i], f);
        load_w<WT, W>(w, (int64_t)c * W, 1.f, wv);
        load_w<WT, W>(bias, (int64_t)c * W, 0.f, bv);
#pragma unroll
        for (int u = 0; u < W; ++u) f[u] = fmaf((f[u] - m) * r, wv[u], bv[u]);
        __stcs(yr + c, pack<E>(f));
    }
}

template <typename E, typename WT>
__global__ void __launch_bounds__(256) norm_stream(const E* x, const WT* __restrict__ w,
                                                   const WT* __restrict__ bias, float eps, E* y,
                                                   float* __restrict__ mean, float* __restrict__ rstd, int64_t rows,
                                                   int64_t width) {
    __shared__ float red[kMaxWarps];
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const E* xr = x + row * width;
        E* yr = y + row * width;
        const float inv = 1.f / (float)width;
        float s = 0.f;
        for (int64_t c = tid; c < width; c += 256) s += to_f(xr[c]);
        const float m = row_sum<256>(s, red, tid) * inv;
        s = 0.f;
        for (int64_t c = tid; c < width; c += 256) {
            const float d = to_f(xr[c]) - m;
            s = fmaf(d, d, s);
        }
        const float r = rsqrtf(row_sum<256>(s, red, tid) * inv + eps);
        if (tid == 0) {
            if (mean) mean[row] = m;
            if (rstd) rstd[row] = r;
        }
        for (int64_t c = tid; c < width; c += 256)
            yr[c] = from_f<E>(fmaf((to_f(xr[c]) - m) * r, w ? to_f(w[c]) : 1.f, bias ? to_f(bias[c]) : 0.f));
    }
}

// --------------------------------------------------------------- backward
// A CTA's threads own the row's vectors (IT each) and walk R rows at a time,
// so that 2 R IT loads a thread are in flight before a barrier; the sums of dw
// and db stay in registers until the end.
template <typename E, typename WT, int IT, int R, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_back_rows(const E* dy, const E* x,
                                                       const WT* __restrict__ w, const float* __restrict__ mean,
                                                       const float* __restrict__ rstd, E* gx,
                                                       float* __restrict__ part, int64_t rows, int width, bool want_w,
                                                       bool want_b) {
    constexpr int W = Vec<E>::W;
    __shared__ float red[2][MAXT / 32][2 * R];
    const int tid = threadIdx.x, nt = blockDim.x, nw = nt / 32, nv = width / W;
    float gw[IT][W], gb[IT][W], wv[IT][W];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = tid + nt * i;
#pragma unroll
        for (int u = 0; u < W; ++u) gw[i][u] = gb[i][u] = 0.f, wv[i][u] = 0.f;
        if (c < nv) load_w<WT, W>(w, (int64_t)c * W, 1.f, wv[i]);
    }
    const float inv = 1.f / (float)width;
    int flip = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < rows; r0 += (int64_t)gridDim.x * R, flip ^= 1) {
        uint4 xr[R][IT], dr[R][IT];
        float m[R], rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool there = r0 + r < rows;
            m[r] = there ? mean[r0 + r] : 0.f;
            rs[r] = there ? rstd[r0 + r] : 0.f;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = tid + nt * i;
                const bool in = there && c < nv;
                xr[r][i] = in ? __ldcs(reinterpret_cast<const uint4*>(x + (r0 + r) * width) + c) : make_uint4(0, 0, 0, 0);
                dr[r][i] = in ? __ldcs(reinterpret_cast<const uint4*>(dy + (r0 + r) * width) + c) : make_uint4(0, 0, 0, 0);
            }
        }
        float s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[2 * r] = s[2 * r + 1] = 0.f;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                float xf[W], df[W];
                unpack<E>(xr[r][i], xf);
                unpack<E>(dr[r][i], df);
#pragma unroll
                for (int u = 0; u < W; ++u) {
                    const float xh = (xf[u] - m[r]) * rs[r], a = df[u] * wv[i][u];
                    s[2 * r] += a;
                    s[2 * r + 1] = fmaf(a, xh, s[2 * r + 1]);
                    gw[i][u] = fmaf(df[u], xh, gw[i][u]);
                    gb[i][u] += df[u];
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2 * R; ++e) {
            s[e] = warp_sum(s[e]);
            if (tid % 32 == 0) red[flip][tid / 32][e] = s[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2 * R; ++e) {
            s[e] = 0.f;
            for (int k = 0; k < nw; ++k) s[e] += red[flip][k][e];
            s[e] *= inv;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r0 + r >= rows) break;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = tid + nt * i;
                if (c >= nv) continue;
                float xf[W], df[W];
                unpack<E>(xr[r][i], xf);
                unpack<E>(dr[r][i], df);
#pragma unroll
                for (int u = 0; u < W; ++u) {
                    const float xh = (xf[u] - m[r]) * rs[r];
                    xf[u] = rs[r] * (df[u] * wv[i][u] - s[2 * r] - xh * s[2 * r + 1]);
                }
                __stcs(reinterpret_cast<uint4*>(gx + (r0 + r) * width) + c, pack<E>(xf));
            }
        }
    }
    float* pw = part + (int64_t)blockIdx.x * 2 * width;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = tid + nt * i;
        if (c >= nv) continue;
#pragma unroll
        for (int u = 0; u < W; ++u) {
            if (want_w) pw[c * W + u] = gw[i][u];
            if (want_b) pw[width + c * W + u] = gb[i][u];
        }
    }
}

// Streaming form: the two row sums first, then dx and the column sums.
template <typename E, typename WT>
__global__ void __launch_bounds__(256) norm_back_sums(const E* dy, const E* x,
                                                      const WT* __restrict__ w, const float* __restrict__ mean,
                                                      const float* __restrict__ rstd, float2* __restrict__ sums,
                                                      int64_t rows, int64_t width) {
    __shared__ float red[kMaxWarps];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float m = mean[row], r = rstd[row];
        float s1 = 0.f, s2 = 0.f;
        for (int64_t c = threadIdx.x; c < width; c += 256) {
            const float a = to_f(dy[row * width + c]) * (w ? to_f(w[c]) : 1.f);
            s1 += a;
            s2 = fmaf(a, (to_f(x[row * width + c]) - m) * r, s2);
        }
        s1 = row_sum<256>(s1, red, threadIdx.x);
        s2 = row_sum<256>(s2, red, threadIdx.x);
        if (threadIdx.x == 0) sums[row] = make_float2(s1 / (float)width, s2 / (float)width);
    }
}
// 32 columns x 8 row lanes a CTA; blockIdx.y takes every gridDim.y-th group of rows.
template <typename E, typename WT>
__global__ void __launch_bounds__(256) norm_back_cols(const E* dy, const E* x,
                                                      const WT* __restrict__ w, const float* __restrict__ mean,
                                                      const float* __restrict__ rstd, const float2* __restrict__ sums,
                                                      E* gx, float* __restrict__ part, int64_t rows,
                                                      int64_t width, bool want_w, bool want_b) {
    __shared__ float red[2][8][33];
    const int lx = threadIdx.x % 32, ly = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lx;
    float gw = 0.f, gb = 0.f;
    if (c < width) {
        const float wv = w ? to_f(w[c]) : 1.f;
        for (int64_t row = (int64_t)blockIdx.y * 8 + ly; row < rows; row += (int64_t)gridDim.y * 8) {
            const float m = mean[row], r = rstd[row], d = to_f(dy[row * width + c]);
            const float xh = (to_f(x[row * width + c]) - m) * r;
            const float2 s = sums[row];
            gx[row * width + c] = from_f<E>(r * (d * wv - s.x - xh * s.y));
            gw = fmaf(d, xh, gw);
            gb += d;
        }
    }
    red[0][ly][lx] = gw;
    red[1][ly][lx] = gb;
    __syncthreads();
    if (ly < 2 && c < width && (ly ? want_b : want_w)) {
        float s = 0.f;
        for (int i = 0; i < 8; ++i) s += red[ly][i][lx];
        part[((int64_t)blockIdx.y * 2 + ly) * width + c] = s;
    }
}

// part [n][2][width] -> gweight, gbias: 32 columns x 8 lanes over n, in a
// fixed order.
template <typename WT>
__global__ void __launch_bounds__(256) norm_back_join(const float* __restrict__ part, int n, int64_t width,
                                                      WT* __restrict__ gw, WT* __restrict__ gb) {
    __shared__ float red[8][33];
    WT* out = blockIdx.y ? gb : gw;
    if (!out) return;
    const int lx = threadIdx.x % 32, ly = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lx;
    float s = 0.f;
    if (c < width)
#pragma unroll 4
        for (int i = ly; i < n; i += 8) s += part[((int64_t)i * 2 + blockIdx.y) * width + c];
    red[ly][lx] = s;
    __syncthreads();
    if (ly == 0 && c < width) {
        s = 0.f;
        for (int i = 0; i < 8; ++i) s += red[i][lx];
        out[c] = from_f<WT>(s);
    }
}

constexpr int kBackGrid = 304;  // row CTAs of the backward: two an SM (152 SMs)

template <typename E>
bool vectors_fit(int64_t width, int64_t most) {
    return width % Vec<E>::W == 0 && width / Vec<E>::W <= most;
}

template <typename E, typename WT>
cudaError_t norm_fwd(const NormArgs& a, cudaStream_t st) {
    const E* x = static_cast<const E*>(a.x);
    const WT* w = static_cast<const WT*>(a.weight);
    const WT* b = static_cast<const WT*>(a.bias);
    E* y = static_cast<E*>(a.y);
    const int64_t nv = a.width / Vec<E>::W;
    auto go = [&](auto* kernel, int tpr, int rpc) {
        kernel<<<(unsigned)((a.rows + rpc - 1) / rpc), tpr * rpc, 0, st>>>(x, w, b, a.eps, y, a.mean, a.rstd, a.rows,
                                                                          (int)a.width);
        return cudaGetLastError();
    };
    if (vectors_fit<E>(a.width, 4096)) {
        if (nv <= 32) return go(norm_rows<E, WT, 32, 1>, 32, 4);
        if (nv <= 64) return go(norm_rows<E, WT, 32, 2>, 32, 4);
        if (nv <= 128) return go(norm_rows<E, WT, 32, 4>, 32, 4);
        if (nv <= 256) return go(norm_rows<E, WT, 32, 8>, 32, 4);
        if (nv <= 1024) return go(norm_rows<E, WT, 256, 4>, 256, 1);
        return go(norm_rows<E, WT, 1024, 4>, 1024, 1);
    }
    norm_stream<E, WT><<<(unsigned)(a.rows < 4 * 2048 ? a.rows : 4 * 2048), 256, 0, st>>>(x, w, b, a.eps, y, a.mean, a.rstd,
                                                                                         a.rows, a.width);
    return cudaGetLastError();
}

int back_groups(int64_t rows) {
    const int64_t want = (rows + 3) / 4;
    return (int)(want < kBackGrid ? want : kBackGrid);
}

template <typename E, typename WT>
cudaError_t norm_bwd(const NormArgs& a, void* ws, cudaStream_t st) {
    const E* x = static_cast<const E*>(a.x);
    const E* dy = static_cast<const E*>(a.dy);
    const WT* w = static_cast<const WT*>(a.weight);
    E* gx = static_cast<E*>(a.gx);
    float2* sums = static_cast<float2*>(ws);
    const int n = back_groups(a.rows);
    float* part = reinterpret_cast<float*>(sums + a.rows);
    const bool ww = a.gweight, wb = a.gbias;
    if (vectors_fit<E>(a.width, 2048)) {
        const int nv = (int)(a.width / Vec<E>::W);
        auto go = [&](auto* kernel, int it) {
            const int nt = ((nv + it - 1) / it + 31) / 32 * 32;
            kernel<<<n, nt, 0, st>>>(dy, x, w, a.mean, a.rstd, gx, part, a.rows, (int)a.width, ww, wb);
        };
        if (nv <= 256)
            go(norm_back_rows<E, WT, 1, 4, 256>, 1);
        else if (nv <= 1024)
            go(norm_back_rows<E, WT, 2, 2, 512>, 2);
        else
            go(norm_back_rows<E, WT, 2, 1, 1024>, 2);
    } else {
        norm_back_sums<E, WT><<<(unsigned)(a.rows < 8192 ? a.rows : 8192), 256, 0, st>>>(dy, x, w, a.mean, a.rstd, sums,
                                                                                        a.rows, a.width);
        norm_back_cols<E, WT><<<dim3((unsigned)((a.width + 31) / 32), n), 256, 0, st>>>(
            dy, x, w, a.mean, a.rstd, sums, gx, part, a.rows, a.width, ww, wb);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!ww && !wb)) return e;
    norm_back_join<WT><<<dim3((unsigned)((a.width + 31) / 32), 2), 256, 0, st>>>(
        part, n, a.width, static_cast<WT*>(a.gweight), static_cast<WT*>(a.gbias));
    return cudaGetLastError();
}

// Calls f with null pointers of the tensor and the weight type.
template <typename F>
cudaError_t by_types(const NormArgs& a, F f) {
    auto with = [&](auto* e) {
        using E = std::remove_pointer_t<decltype(e)>;
        if (a.wtype == CSSD_F32) return f(e, static_cast<float*>(nullptr));
        return f(e, static_cast<E*>(nullptr));
    };
    if (a.xtype == CSSD_BF16) return with(static_cast<__nv_bfloat16*>(nullptr));
    if (a.xtype == CSSD_F16) return with(static_cast<__half*>(nullptr));
    return with(static_cast<float*>(nullptr));
}

}  // namespace

size_t layernorm_backward_workspace_bytes(int64_t rows, int64_t width) {
    return sizeof(float) * (2 * (size_t)rows + (size_t)back_groups(rows) * 2 * (size_t)width);
}

cudaError_t launch_layernorm(const NormArgs& a, cudaStream_t st) {
    return by_types(a, [&](auto* e, auto* w) {
        return norm_fwd<std::remove_pointer_t<decltype(e)>, std::remove_pointer_t<decltype(w)>>(a, st);
    });
}
cudaError_t launch_layernorm_backward(const NormArgs& a, void* ws, cudaStream_t st) {
    return by_types(a, [&](auto* e, auto* w) {
        return norm_bwd<std::remove_pointer_t<decltype(e)>, std::remove_pointer_t<decltype(w)>>(a, ws, st);
    });
}

}  // namespace cssd
