// Helpers shared by the gated-delta-rule kernels: element types, the decays
// of one chunk, and the inverse of its unit lower triangular matrix.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

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

// Programmatic dependent launch: let the kernel behind this one in the stream
// (if it was launched so) start; wait until the kernel before it has ended.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Dynamic shared memory of kernel F, allowed once per device (`bytes` is the
// most that any launch of F asks for).
template <auto* F>
inline cudaError_t allow(uint32_t bytes) {
    static std::atomic<uint64_t> done[2] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool track = dev >= 0 && dev < 128;
    if (track && (done[dev / 64].load(std::memory_order_acquire) >> (dev % 64) & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(F), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && track) done[dev / 64].fetch_or(1ull << (dev % 64), std::memory_order_release);
    return e;
}

// A sum kept as two floats, value and what its rounding left.
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 add(Sum2 a, Sum2 b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float h = s + e;
    return {h, e - (h - s)};
}
__device__ __forceinline__ float exp_of(Sum2 s) { return expf(s.hi) * (1.f + (isfinite(s.hi) ? s.lo : 0.f)); }

// The decays of one chunk, from the running sum G_i of its log decays.  The
// sums are kept as two floats, because exp(G_i - G_j) needs the difference of
// two sums to an absolute 1e-7 while the sums themselves reach hundreds.
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
    Sum2 s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        float gv = 0.f, bv = 0.f;
        if (i < n) {
            gv = g[i * stride];
            bv = beta[i * stride];
        }
        d.beta[i] = bv;
        s[e] = {gv < -1000.f ? -1000.f : gv, 0.f};
    }
    s[1] = add(s[0], s[1]);
    Sum2 tot = s[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum2 up = {__shfl_up_sync(0xffffffffu, tot.hi, o), __shfl_up_sync(0xffffffffu, tot.lo, o)};
        if (lane >= o) tot = add(up, tot);
    }
    Sum2 before = {__shfl_up_sync(0xffffffffu, tot.hi, 1), __shfl_up_sync(0xffffffffu, tot.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const Sum2 end = {__shfl_sync(0xffffffffu, tot.hi, 31), __shfl_sync(0xffffffffu, tot.lo, 31)};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        const Sum2 G = add(before, s[e]);
        d.hi[i] = G.hi;
        d.lo[i] = G.lo;
        d.in[i] = exp_of(G);
        d.out[i] = exp_of(add(end, {-G.hi, -G.lo}));
        if (i == C - 1) d.all = d.in[i];
    }
}

// exp(G_i - G_j); the caller masks the pairs with i < j.
__device__ __forceinline__ float decay_between(const Decays& d, int i, int j) {
    return expf((d.hi[i] - d.hi[j]) + (d.lo[i] - d.lo[j]));
}

// Sums y over the SPLIT neighbouring lanes that hold parts of it; lane l of
// them gets rows l R / SPLIT and on of the R, in y's first.
template <int SPLIT, int R>
__device__ __forceinline__ void join(float (&y)[R][4], int l) {
    if (SPLIT == 4) {
        const bool high = l & 2;
#pragma unroll
        for (int a = 0; a < R / 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float other = __shfl_xor_sync(0xffffffffu, high ? y[a][i] : y[a + R / 2][i], 2);
                y[a][i] = (high ? y[a + R / 2][i] : y[a][i]) + other;
            }
    }
    constexpr int H = SPLIT == 4 ? R / 4 : R / 2;
    const bool odd = l & 1;
#pragma unroll
    for (int a = 0; a < H; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? y[a][i] : y[a + H][i], 1);
            y[a][i] = (odd ? y[a + H][i] : y[a][i]) + other;
        }
}

// y += rows r0 .. r0 + 3 of A times columns c0 .. c0 + 3 of B, k from `from` on
// in steps of four below `to`: a quarter of the product.
__device__ __forceinline__ void quarter_product(float (&y)[4][4], const float* A, int lda, const float* B, int ldb, int r0,
                                                int c0, int from, int to) {
#pragma unroll 2
    for (int m = from; m < to; m += 4) {
        const float4 t = *reinterpret_cast<const float4*>(B + m * ldb + c0);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const float v = A[(r0 + a) * lda + m];
            y[a][0] = fmaf(v, t.x, y[a][0]);
            y[a][1] = fmaf(v, t.y, y[a][1]);
            y[a][2] = fmaf(v, t.z, y[a][2]);
            y[a][3] = fmaf(v, t.w, y[a][3]);
        }
    }
}

// (I + a)^-1 in place of the strictly lower triangular a (64 x 64, row stride
// LD, fp32, in shared memory, 16-byte aligned rows), by 256 threads: the four
// 16 x 16 blocks on the diagonal by forward substitution, one column a thread,
// then two rounds of
//     [L11 0; A21 L22]^-1 = [T11 0; -T22 A21 T11 T22],
// 4 x 4 outputs to four neighbouring lanes that share the sum: 2 bytes of
// shared memory a multiply-add, which is what bounds it.  `w` is kInverseScratch
// floats, 16-byte aligned.  All threads call it; the result is complete after
// its last barrier.  The upper triangle has to be zeros and stays so.
constexpr int kInverseScratch = 32 * 36;
template <int LD>
__device__ void tri_inverse_in_place(float* a, float* w, int tid) {
    if (tid < 64) {
        const int b = tid >> 4, j = tid & 15;
        float* ab = a + (b * 16) * LD + b * 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == j ? 1.f : 0.f, s2 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 v = *reinterpret_cast<const float4*>(ab + i * LD + m);
                s = fmaf(-v.x, x[m], s);
                if (m + 1 < i) s2 = fmaf(-v.y, x[m + 1], s2);
                if (m + 2 < i) s = fmaf(-v.z, x[m + 2], s);
                if (m + 3 < i) s2 = fmaf(-v.w, x[m + 3], s2);
            }
            x[i] = i < j ? 0.f : s + s2;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) ab[i * LD + j] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int half = 16; half <= 32; half *= 2) {
        // a warp: two rows of four tiles, so that the lanes' words of A and rows of
        // B meet no bank twice
        const int l = tid & 3, t = tid >> 2, LW = half + 4;
        const int c0 = 4 * ((t >> 1 & 3) + (half == 32 ? t >> 1 & 4 : 0));
        const int r0 = 4 * ((t & 1) + (half == 32 ? t >> 3 & 6 : t >> 2 & 2));
        const int p = half == 32 ? 0 : t >> 4;
        const bool on = p < C / (2 * half);  // (whole warps)
        float* a21 = a + (2 * p + 1) * half * LD + 2 * p * half;
        const float* t11 = a + 2 * p * half * LD + 2 * p * half;
        const float* t22 = a + (2 * p + 1) * half * LD + (2 * p + 1) * half;
        float* wp = w + p * half * LW;
        if (on) {  // w = A21 T11
            float y[4][4] = {};
            quarter_product(y, a21, LD, t11, LD, r0, c0, c0 + l, half);
            join<4>(y, l);
            *reinterpret_cast<float4*>(wp + (r0 + l) * LW + c0) = make_float4(y[0][0], y[0][1], y[0][2], y[0][3]);
        }
        __syncthreads();
        if (on) {  // T21 = -T22 w, over A21
            float y[4][4] = {};
            quarter_product(y, t22, LD, wp, LW, r0, c0, l, r0 + 4);
            join<4>(y, l);
            *reinterpret_cast<float4*>(a21 + (r0 + l) * LD + c0) = make_float4(-y[0][0], -y[0][1], -y[0][2], -y[0][3]);
        }
        __syncthreads();
    }
}

}  // namespace delta
}  // namespace cssd
