// Helpers shared by the gated-delta-rule kernels: element types, the decays
// of one chunk, and the inverse of its unit lower triangular matrix.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cssd_internal.h"

namespace cssd {
namespace delta {

constexpr int C = 64;  // tokens per chunk

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Tokens of batch row b that are there (lens may be null; values outside
// [0, T] count as the nearer bound).
__device__ __forceinline__ int row_len(const int* lens, int b, int T) {
    return lens ? min(max(lens[b], 0), T) : T;
}

// The decays of one chunk, from the running sum G_i of its log decays.  The
// sum is taken in double and kept as two floats, because exp(G_i - G_j) needs
// the difference of two sums to an absolute 1e-7 while the sums themselves
// reach hundreds.
struct Decays {
    float hi[C], lo[C];  // G_i as hi + lo
    float in[C];         // exp(G_i): from the chunk's start through token i
    float out[C];        // exp(G_end - G_i): from token i to the chunk's end
    float beta[C];
    float all;           // exp(G_end)
};

// One warp; tokens at or past `n` (of C) count as g = 0, beta = 0.  g and beta
// point at the chunk's first token, `stride` elements between tokens.  A log
// decay of -inf (a full reset) is taken as -1000, whose exponential is 0 too,
// so that differences of sums stay numbers; NaN passes through.
__device__ __forceinline__ void chunk_decays(Decays& d, const float* g, const float* beta, int64_t stride, int n,
                                             int lane) {
    double s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        float gv = 0.f, bv = 0.f;
        if (i < n) {
            gv = g[i * stride];
            bv = beta[i * stride];
        }
        gv = gv < -1000.f ? -1000.f : gv;
        d.beta[i] = bv;
        s[e] = (double)gv;
    }
    s[1] += s[0];
    double tot = s[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, tot, o);
        if (lane >= o) tot += up;
    }
    double before = __shfl_up_sync(0xffffffffu, tot, 1);
    if (lane == 0) before = 0.0;
    const double end = __shfl_sync(0xffffffffu, tot, 31);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        const double G = before + s[e];
        const float hi = (float)G, lo = (float)(G - (double)hi);
        const double r = end - G;
        const float rh = (float)r, rl = (float)(r - (double)rh);
        d.hi[i] = hi;
        d.lo[i] = isfinite(hi) ? lo : 0.f;
        d.in[i] = expf(hi) * (1.f + d.lo[i]);
        d.out[i] = expf(rh) * (1.f + (isfinite(rh) ? rl : 0.f));
        if (i == C - 1) d.all = d.in[i];
    }
}

// exp(G_i - G_j); the caller masks the pairs with i < j.
__device__ __forceinline__ float decay_between(const Decays& d, int i, int j) {
    return expf((d.hi[i] - d.hi[j]) + (d.lo[i] - d.lo[j]));
}

// t = (I + a)^-1 for the strictly lower triangular a (64 x 64, row stride
// LD, fp32, in shared memory), by 256 threads: the four 16 x 16 blocks on the
// diagonal by forward substitution, one column a thread, then two rounds of
//   [L11 0; A21 L22]^-1 = [T11 0; -T22 A21 T11 T22].
// `w` is 32 x 32 floats of scratch.  All threads call it; t is complete after
// its last barrier.  t's upper triangle is written as zeros.
template <int LD>
__device__ void tri_inverse(const float* a, float* t, float* w, int tid) {
    for (int e = tid; e < C * C; e += 256) {
        const int i = e / C, j = e % C;
        if ((j >> 4) > (i >> 4)) t[i * LD + j] = 0.f;
    }
    if (tid < 64) {
        const int b = tid >> 4, j = tid & 15;
        const float* ab = a + (b * 16) * LD + b * 16;
        float* tb = t + (b * 16) * LD + b * 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == j ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; ++m) s = fmaf(-ab[i * LD + m], x[m], s);
            x[i] = i < j ? 0.f : s;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) tb[i * LD + j] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int half = 16; half <= 32; half *= 2) {
        const int pairs = C / (2 * half), per = half * half;
        for (int e = tid; e < pairs * per; e += 256) {  // w = A21 T11
            const int p = e / per, r = (e % per) / half, c = e % half;
            const float* a21 = a + (2 * p + 1) * half * LD + 2 * p * half;
            const float* t11 = t + 2 * p * half * LD + 2 * p * half;
            float s = 0.f;
#pragma unroll 8
            for (int m = 0; m < half; ++m) s = fmaf(a21[r * LD + m], t11[m * LD + c], s);
            w[e] = s;
        }
        __syncthreads();
        for (int e = tid; e < pairs * per; e += 256) {  // T21 = -T22 w
            const int p = e / per, r = (e % per) / half, c = e % half;
            const float* t22 = t + (2 * p + 1) * half * LD + (2 * p + 1) * half;
            float s = 0.f;
#pragma unroll 8
            for (int m = 0; m < half; ++m) s = fmaf(-t22[r * LD + m], w[p * per + m * half + c], s);
            t[((2 * p + 1) * half + r) * LD + 2 * p * half + c] = s;
        }
        __syncthreads();
    }
}

}  // namespace delta
}  // namespace cssd
