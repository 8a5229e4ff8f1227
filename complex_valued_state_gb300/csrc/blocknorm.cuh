#pragma once

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
//
// Measured, 8192 x 1536 bf16 (device time): add with an fp32 residual 25 us (151 MB: 5.9 TB/s), its gradients 41 and 4
// for the join (227 MB: 5.0 TB/s with it); gated by heads of 64 17 us (76 MB: 4.4 TB/s; issue 76 % busy: the gate's
// exponential and reciprocal), gradients over whole rows 32 and 4 (126 MB: 3.5 TB/s).  Widths that are no whole
// 16-byte vectors, rows too wide for the registers or the ring, and the gradients of narrow groups that are no power of
// two of vectors, take the streaming kernels, which read a row again from the caches for each sum: 47, 93, 102 and
// 117 us for these cases.

#include <initializer_list>
#include <type_traits>

#include "cssd_internal.h"
#include "delta_common.cuh"
#include "tcgen05.cuh"

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
// 1 / (1 + e^-z), for tensors of type E.  The quick exponential of x is off by up to 2 + 1.2 |x| steps of 2^-23 (the
// rounding of x log2(e) grows with x), and with it the sigmoid far below 0, where it is about e^z: results were off by
// 62 2^-24 at z = -80, by 17 at -20, by 5 above 0.  That is 2^-16 at most before e^-z overflows, far below half a
// step of 16-bit results; float tensors take the full exponential, 5 2^-24 for every z (8192 x 1536, fp32, groups of 64:
// 24.9 us against 22.8; with a full division too 26.9).  The quotient is quick for both (2 steps of 2^-23; 0 below -87).
template <typename E>
__device__ __forceinline__ float sigmoid(float z) {
    return __fdividef(1.f, 1.f + (std::is_same_v<E, float> ? expf(-z) : __expf(-z)));
}

// --------------------------------------------------------------- vectors
template <typename E>
struct Vec {
    static constexpr int W = 16 / sizeof(E);
};
// W values of type T from 16-byte aligned memory (W sizeof(T) is a multiple of 16), and back.
template <typename T, int W>
__device__ __forceinline__ void load(const T* p, float (&f)[W]) {
    static_assert(W * sizeof(T) % 16 == 0, "whole vectors");
    alignas(16) T t[W];
#pragma unroll
    for (int i = 0; i < (int)(W * sizeof(T) / 16); ++i) reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = to_f(t[i]);
}
template <typename T, int W>
__device__ __forceinline__ void load_once(const T* p, float (&f)[W]) {
    alignas(16) T t[W];
#pragma unroll
    for (int i = 0; i < (int)(W * sizeof(T) / 16); ++i) reinterpret_cast<uint4*>(t)[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = to_f(t[i]);
}
template <typename E>
__device__ __forceinline__ void unpack(const uint4& raw, float (&f)[Vec<E>::W]) {
    alignas(16) E t[Vec<E>::W];
    *reinterpret_cast<uint4*>(t) = raw;
#pragma unroll
    for (int i = 0; i < Vec<E>::W; ++i) f[i] = to_f(t[i]);
}
template <typename T, int W>
__device__ __forceinline__ void store(T* p, const float (&f)[W]) {
    alignas(16) T t[W];
#pragma unroll
    for (int i = 0; i < W; ++i) t[i] = from_f<T>(f[i]);
#pragma unroll
    for (int i = 0; i < (int)(W * sizeof(T) / 16); ++i) __stcs(reinterpret_cast<uint4*>(p) + i, reinterpret_cast<uint4*>(t)[i]);
}
template <typename T, int W>
__device__ __forceinline__ void load_or(const T* p, int64_t at, float other, float (&f)[W]) {
    if (p) return load<T, W>(p + at, f);
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = other;
}

// Sum over TPR neighbouring lanes (TPR <= 32: a power of two), or a CTA's threads.
template <int TPR>
__device__ __forceinline__ float lanes_sum(float v, float* red, int tid) {
    if constexpr (TPR > 32)
        return team_sum<TPR>(v, red, tid);
    else {
#pragma unroll
        for (int o = TPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
}

// The vectors that a thread has of a row: TPR threads, IT vectors each.  `HEADS`: rows as narrow as a head too,
// and none beyond 1024 vectors.
template <bool HEADS, typename F>
cudaError_t by_vectors(int64_t nv, F f) {
    using std::integral_constant;
#define CSSD_ROWS(t, i) f(integral_constant<int, t>(), integral_constant<int, i>())
    if constexpr (HEADS) {
        if (nv <= 8) return CSSD_ROWS(8, 1);
        if (nv <= 16) return CSSD_ROWS(16, 1);
    }
    if (nv <= 32) return CSSD_ROWS(32, 1);
    if (nv <= 64) return CSSD_ROWS(32, 2);
    if (nv <= 128) return CSSD_ROWS(32, 4);
    if (nv <= 192) return CSSD_ROWS(32, 6);
    if constexpr (!HEADS)
        if (nv > 1024) return CSSD_ROWS(1024, 4);
    return CSSD_ROWS(256, 4);
#undef CSSD_ROWS
}
template <typename E>
bool vectors_fit(int64_t width, int64_t most) {
    return width % Vec<E>::W == 0 && width / Vec<E>::W <= most;
}

// --------------------------------------------------------------- the gradients' ring
// Rows come by bulk copies into a ring in shared memory, kStages - 1 rows ahead: G warps a row, so 8 / G rows at
// a time in a CTA; registers hold the column sums alone, and the copies in flight are what keeps the memory
// busy.  The warps add up their column sums at the end.  Two stages: with three the gated gradients took 35.9 us
// against 32.1 and the others the same; 16 warps a CTA 50 us, three CTAs an SM 39.
constexpr int kRowWarps = 8;
constexpr int kStages = 2;
constexpr long long kNormWait = 4000000000LL;  // ~2 s at 2 GHz

template <int G>
__device__ __forceinline__ void group_barrier(int group) {
    if constexpr (G == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * G) : "memory");
}
// The sums of two values over a group's threads.
template <int G>
__device__ __forceinline__ float2 group_sums(float a, float b, float (*red)[2], int group, int warp, int lane) {
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (G > 1) {
        if (lane == 0) red[warp][0] = a, red[warp][1] = b;
        group_barrier<G>(group);
        a = b = 0.f;
#pragma unroll
        for (int e = 0; e < G; ++e) a += red[group * G + e][0], b += red[group * G + e][1];
    } else {
        __syncwarp();
    }
    return make_float2(a, b);
}
// A vector of the caller's as floats in shared memory (`other` where there is none).
__device__ __forceinline__ void spread(float* to, const void* v, bool wide, int xtype, float other, int64_t from, int n, int tid, int nt) {
    for (int c = tid; c < n; c += nt) {
        float f = other;
        if (v) {
            if (wide)
                f = static_cast<const float*>(v)[from + c];
            else if (xtype == CSSD_BF16)
                f = to_f(static_cast<const __nv_bfloat16*>(v)[from + c]);
            else
                f = to_f(static_cast<const __half*>(v)[from + c]);
        }
        to[c] = f;
    }
}
// One column sum of all groups, one group after another, into part (K of them a CTA).
template <int W, int IT, int G>
__device__ __forceinline__ void join_groups(const float (&v)[IT][W], float* sum, float* part, bool wanted, int width, int group, int gt,
                                            int tid) {
    constexpr int TG = 32 * G;
    for (int e = 0; e < kRowWarps / G; ++e) {
        if (group == e)
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int u = 0; u < W; ++u) {
                    float* at = sum + (u * IT + i) * TG + gt;  // (threads side by side)
                    *at = (e ? *at : 0.f) + v[i][u];
                }
        __syncthreads();
    }
    if (wanted)
        for (int c = tid; c < width; c += 32 * kRowWarps) {
            const int x = c / W, u = c % W;
            part[c] = sum[(u * IT + x / TG) * TG + x % TG];
        }
    __syncthreads();
}

// Calls f(G, IT) for rows of nv vectors of which a stage of the ring takes `bytes` and the vectors in shared
// memory `vec`: two CTAs an SM where that goes, else one; false if neither does.
struct RingPlan {
    int G, IT;
    size_t smem;
};
inline bool plan_ring(int64_t nv, int W, size_t bytes, size_t vec, RingPlan& p) {
    for (size_t most : {(size_t)112 << 10, (size_t)220 << 10})
        for (int G = 1; G <= 8; G *= 2) {
            int IT = (int)((nv + 32 * G - 1) / (32 * G));
            if (IT > 3) continue;
            if (G > 1 && IT == 1) IT = 2;  // (such a row has G = 1, but for its bytes)
            const size_t ring = (size_t)(kRowWarps / G) * kStages * bytes + vec, sums = sizeof(float) * 32 * G * IT * W;
            const size_t smem = ring > sums ? ring : sums;
            if (smem <= most) {
                p = {G, IT, smem};
                return true;
            }
        }
    return false;
}
template <typename F>
cudaError_t by_plan(const RingPlan& p, F f) {
    using std::integral_constant;
    auto with = [&](auto g) {
        if constexpr (decltype(g)::value == 1)
            if (p.IT == 1) return f(g, integral_constant<int, 1>());
        if (p.IT == 2) return f(g, integral_constant<int, 2>());
        return f(g, integral_constant<int, 3>());
    };
    if (p.G == 1) return with(integral_constant<int, 1>());
    if (p.G == 2) return with(integral_constant<int, 2>());
    if (p.G == 4) return with(integral_constant<int, 4>());
    return with(integral_constant<int, 8>());
}

// --------------------------------------------------------------- column sums
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

// part [n][k][width] -> the k vectors (null: not wanted): 32 columns x 32 lanes over n, in a fixed order.
template <typename W>
struct Vectors {
    W *a, *b, *c;
};
template <typename W>
__global__ void __launch_bounds__(1024) join_columns(const float* part, int n, int64_t width, Vectors<W> out) {
    __shared__ float red[32][33];
    W* to = blockIdx.y == 0 ? out.a : blockIdx.y == 1 ? out.b : out.c;
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
    return cudaLaunchKernelEx(&cfg, join_columns<W>, part, n, width, Vectors<W>{a, b, c});
}

// Calls f with a null pointer of the tensors' type or of float.
template <typename E, typename F>
cudaError_t or_float(bool wide, E* e, F f) {
    if constexpr (!std::is_same_v<E, float>)
        if (!wide) return f(e);
    return f(static_cast<float*>(nullptr));
}
template <typename P>
using To = std::remove_pointer_t<P>;

}  // namespace
}  // namespace cssd
