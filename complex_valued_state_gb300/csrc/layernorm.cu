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
//
// Measured, bf16: 8192 x 1536 forward 10.3 us (4.9 TB/s of tensors that L2
// partly holds), gradients 22 us (3.4 TB/s: the CTAs' 304 partial sums and the
// kernel that joins them take 4 us of it); gradients of 65536 x 2048 165 us
// (4.9 TB/s).  From a cold L2 8192 x 1536 takes 20 and 30 us, and the streaming
// kernels, which read 2 bytes a lane and in the gradients everything twice, 30 and
// 50 us for 8192 x 1001.

#include <type_traits>

#include "cssd_internal.h"
#include "delta_common.cuh"
#include "pairs.cuh"
#include "tcgen05.cuh"

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
// One row's share of the sums (a: dy w, so sum a and sum a xh) and of the
// column sums, for a vector of the row, two elements an instruction.
// `r2` holds rstd twice, `m2` -mean: the mean is taken off before rstd is
// multiplied on, since x rstd - mean rstd would be off by 2^-24 of mean rstd.
template <typename E>
__device__ __forceinline__ void back_sums(const uint4& xr, const uint4& dr, f2 r2, f2 m2, const f2* wv, f2& s1, f2& s2,
                                          f2 (&gw)[Vec<E>::W / 2], f2 (&gb)[Vec<E>::W / 2]) {
    float xf[Vec<E>::W], df[Vec<E>::W];
    unpack<E>(xr, xf);
    unpack<E>(dr, df);
#pragma unroll
    for (int u = 0; u < Vec<E>::W / 2; ++u) {
        const f2 d = mk2(df[2 * u], df[2 * u + 1]);
        const f2 xh = mul2(add2(mk2(xf[2 * u], xf[2 * u + 1]), m2), r2), a = mul2(d, wv[u]);
        s1 = add2(s1, a);
        s2 = fma2(a, xh, s2);
        gw[u] = fma2(d, xh, gw[u]);
        gb[u] = add2(gb[u], d);
    }
}
// dx of the vector: `t1` and `t2` hold -rstd times the row's two means.
template <typename E>
__device__ __forceinline__ uint4 back_dx(const uint4& xr, const uint4& dr, f2 r2, f2 m2, const f2* wv, f2 t1, f2 t2) {
    float xf[Vec<E>::W], df[Vec<E>::W];
    unpack<E>(xr, xf);
    unpack<E>(dr, df);
#pragma unroll
    for (int u = 0; u < Vec<E>::W / 2; ++u) {
        const f2 xh = mul2(add2(mk2(xf[2 * u], xf[2 * u + 1]), m2), r2);
        const f2 a = mul2(mk2(df[2 * u], df[2 * u + 1]), wv[u]);
        un2(fma2(xh, t2, fma2(a, r2, t1)), xf[2 * u], xf[2 * u + 1]);
    }
    return pack<E>(xf);
}

// G warps a row, IT vectors a thread, rows of x and dy by bulk copies into a
// ring in shared memory, kStages - 1 rows ahead: registers hold the column sums
// alone, and the copies in flight (8 / G groups of warps times the ring) are
// what keeps the memory busy.  The warps add up their column sums at the end.
// 8192 x 1536 bf16: 22 us with the join; rows loaded into registers two at a
// time, as norm_back_rows does, took 30.
constexpr int kRowWarps = 8;
constexpr int kStages = 4;
constexpr long long kNormWait = 4000000000LL;  // ~2 s at 2 GHz

template <int G>
__device__ __forceinline__ void group_barrier(int group) {
    if constexpr (G == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * G) : "memory");
}

template <typename E, typename WT, int IT, int G>
__global__ void __launch_bounds__(32 * kRowWarps, 2)
    norm_back_ring(const E* dy, const E* x, const WT* __restrict__ w, const float* __restrict__ mean,
                   const float* __restrict__ rstd, E* gx, float* __restrict__ part, int64_t rows, int width, bool want_w,
                   bool want_b, unsigned* status) {
    constexpr int W = Vec<E>::W, NG = kRowWarps / G, TG = 32 * G;
    extern __shared__ __align__(128) unsigned char ring[];  // [group][stage][x, dy][width], then the weights
    __shared__ __align__(8) uint64_t full[NG][kStages];
    __shared__ float red[2][kRowWarps][2];
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, group = warp / G, gt = tid % TG, nv = width / W;
    const uint32_t bytes = (uint32_t)width * sizeof(E);
    delta::let_next_start();
    unsigned char* mine = ring + (size_t)group * kStages * 2 * bytes;
    float* sw = reinterpret_cast<float*>(ring + (size_t)NG * kStages * 2 * bytes);
    for (int c = tid; c < width; c += 32 * kRowWarps) sw[c] = w ? to_f(w[c]) : 1.f;
    if (tid == 0) {
        s_gave_up = 0;
        for (int i = 0; i < NG; ++i)
            for (int j = 0; j < kStages; ++j) tc::mbar_init(&full[i][j], 1);
        tc::mbar_fence_init();
    }
    __syncthreads();
    f2 gw[IT][W / 2], gb[IT][W / 2];
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int u = 0; u < W / 2; ++u) gw[i][u] = gb[i][u] = 0;
    const float inv = 1.f / (float)width;
    const int64_t step = (int64_t)gridDim.x * NG, row0 = (int64_t)blockIdx.x * NG + group;
    auto fetch = [&](int64_t k) {  // the group's k-th row
        const int64_t row = row0 + k * step;
        if (row >= rows) return;
        const int st = (int)(k % kStages);
        const uint32_t at = tc::smem_u32(mine) + st * 2 * bytes;
        tc::mbar_arrive_expect_tx(&full[group][st], 2 * bytes);
        tc::bulk_g2s(at, x + row * width, bytes, &full[group][st]);
        tc::bulk_g2s(at + bytes, dy + row * width, bytes, &full[group][st]);
    };
    if (gt == 0)
        for (int k = 0; k < kStages - 1; ++k) fetch(k);
    int64_t k = 0;
    for (int64_t row = row0; row < rows; row += step, ++k) {
        const int st = (int)(k % kStages);
        const float m = mean[row], rs = rstd[row];
        // (a wait that gives up: the row's results are wrong and the status word says so)
        if (!tc::mbar_wait_bounded(&full[group][st], (uint32_t)(k / kStages & 1), kNormWait)) s_gave_up = 1;
        const uint4* xr = reinterpret_cast<const uint4*>(mine + st * 2 * bytes);
        const uint4* dr = reinterpret_cast<const uint4*>(mine + st * 2 * bytes + bytes);
        const f2 r2 = mk2(rs, rs), m2 = mk2(-m, -m);
        f2 p1 = 0, p2 = 0;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = gt + TG * i;
            if (c < nv) back_sums<E>(xr[c], dr[c], r2, m2, reinterpret_cast<const f2*>(sw + c * W), p1, p2, gw[i], gb[i]);
        }
        float s1 = sum2(p1), s2 = sum2(p2);
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if constexpr (G > 1) {
            float(*r)[2] = red[k & 1];
            if (lane == 0) r[warp][0] = s1, r[warp][1] = s2;
            group_barrier<G>(group);
            s1 = s2 = 0.f;
#pragma unroll
            for (int e = 0; e < G; ++e) s1 += r[group * G + e][0], s2 += r[group * G + e][1];
        } else {
            __syncwarp();
        }
        // every thread of the group is past the row before: its stage is free
        if (gt == 0) fetch(k + kStages - 1);
        const float t1 = -rs * s1 * inv, t2 = -rs * s2 * inv;
        uint4* gp = reinterpret_cast<uint4*>(gx + row * width);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = gt + TG * i;
            if (c < nv)
                __stcs(gp + c, back_dx<E>(xr[c], dr[c], r2, m2, reinterpret_cast<const f2*>(sw + c * W), mk2(t1, t1), mk2(t2, t2)));
        }
    }
    if (gt == 0 && s_gave_up)  // no copy may land in shared memory that is no longer this CTA's
        for (int64_t e = k > kStages ? k - kStages : 0; e < k; ++e)
            tc::mbar_wait_bounded(&full[group][e % kStages], (uint32_t)(e / kStages & 1), kNormWait);
    // the groups' column sums, one after another (the copies have all been waited for)
    __syncthreads();
    float* sum = reinterpret_cast<float*>(ring);
    float* pw = part + (int64_t)blockIdx.x * 2 * width;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        for (int e = 0; e < NG; ++e) {
            if (group == e)
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int u = 0; u < W; u += 2) {
                        float v[2];
                        un2(which ? gb[i][u / 2] : gw[i][u / 2], v[0], v[1]);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            float* at = sum + ((u + z) * IT + i) * TG + gt;  // (threads side by side)
                            *at = (e ? *at : 0.f) + v[z];
                        }
                    }
            __syncthreads();
        }
        if (which ? want_b : want_w)
            for (int c = tid; c < width; c += 32 * kRowWarps) {
                const int v = c / W, u = c % W;
                pw[which * width + c] = sum[(u * IT + v / TG) * TG + v % TG];
            }
        __syncthreads();
    }
    if (tid == 0 && s_gave_up && status) atomicOr(status, kStatusNorm);
}

// Rows of more than 768 vectors, three a thread of the ring's 256.  (The ring of
// 16-bit rows leaves one CTA an SM above about 5770 columns already: 8192 rows of
// 5760 take 69 us from a cold L2, of 6144 99.)  A CTA's threads own the row's
// vectors (IT each) and walk R rows at a time, so that 2 R IT loads a thread are
// in flight before a barrier; the sums of dw and db stay in registers until the
// end.  8192 x 8192 bf16 takes 143 us from a cold L2 (1024 threads, 64 registers: the
// 16-bit forms spill 156 to 308 bytes a thread).
template <typename E, typename WT, int IT, int R, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_back_rows(const E* dy, const E* x,
                                                       const WT* __restrict__ w, const float* __restrict__ mean,
                                                       const float* __restrict__ rstd, E* gx,
                                                       float* __restrict__ part, int64_t rows, int width, bool want_w,
                                                       bool want_b) {
    constexpr int W = Vec<E>::W;
    __shared__ float red[2][MAXT / 32][2 * R];
    const int tid = threadIdx.x, nt = blockDim.x, nw = nt / 32, nv = width / W;
    f2 gw[IT][W / 2], gb[IT][W / 2], wv[IT][W / 2];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = tid + nt * i;
        float f[W];
#pragma unroll
        for (int u = 0; u < W; ++u) f[u] = 0.f;
        if (c < nv) load_w<WT, W>(w, (int64_t)c * W, 1.f, f);
#pragma unroll
        for (int u = 0; u < W / 2; ++u) gw[i][u] = gb[i][u] = 0, wv[i][u] = mk2(f[2 * u], f[2 * u + 1]);
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
            f2 p1 = 0, p2 = 0;
            const f2 r2 = mk2(rs[r], rs[r]), m2 = mk2(-m[r], -m[r]);
#pragma unroll
            for (int i = 0; i < IT; ++i)
                if (tid + nt * i < nv) back_sums<E>(xr[r][i], dr[r][i], r2, m2, wv[i], p1, p2, gw[i], gb[i]);
            s[2 * r] = sum2(p1);
            s[2 * r + 1] = sum2(p2);
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
            const f2 r2 = mk2(rs[r], rs[r]), m2 = mk2(-m[r], -m[r]);
            const float t1 = -rs[r] * s[2 * r], t2 = -rs[r] * s[2 * r + 1];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = tid + nt * i;
                if (c < nv)
                    __stcs(reinterpret_cast<uint4*>(gx + (r0 + r) * width) + c,
                           back_dx<E>(xr[r][i], dr[r][i], r2, m2, wv[i], mk2(t1, t1), mk2(t2, t2)));
            }
        }
    }
    float* pw = part + (int64_t)blockIdx.x * 2 * width;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = tid + nt * i;
        if (c >= nv) continue;
#pragma unroll
        for (int u = 0; u < W; u += 2) {
            float v0, v1;
            un2(gw[i][u / 2], v0, v1);
            if (want_w) pw[c * W + u] = v0, pw[c * W + u + 1] = v1;
            un2(gb[i][u / 2], v0, v1);
            if (want_b) pw[width + c * W + u] = v0, pw[width + c * W + u + 1] = v1;
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

// part [n][2][width] -> gweight, gbias: 32 columns x 32 lanes over n, in a
// fixed order.
template <typename WT>
__global__ void __launch_bounds__(1024) norm_back_join(const float* part, int n, int64_t width,
                                                       WT* __restrict__ gw, WT* __restrict__ gb) {
    __shared__ float red[32][33];
    WT* out = blockIdx.y ? gb : gw;
    if (!out) return;
    const int lx = threadIdx.x % 32, ly = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lx;
    float s = 0.f;
    delta::wait_for_previous();  // (nothing of `part` is read before)
    if (c < width)
#pragma unroll 8
        for (int i = ly; i < n; i += 32) s += part[((int64_t)i * 2 + blockIdx.y) * width + c];
    red[ly][lx] = s;
    __syncthreads();
    s = warp_sum(red[lx][ly]);  // column ly, over the lanes
    const int64_t oc = (int64_t)blockIdx.x * 32 + ly;
    if (lx == 0 && oc < width) out[oc] = from_f<WT>(s);
}

constexpr int kBackGrid = 304;  // CTAs of the backward: two an SM (152 SMs)

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

// Partial column sums the backward's kernels may leave (each has a row at least).
int back_groups(int64_t rows) {
    return (int)(rows < kBackGrid ? rows : kBackGrid);
}

template <typename E, typename WT>
cudaError_t norm_bwd(const NormArgs& a, void* ws, cudaStream_t st) {
    const E* x = static_cast<const E*>(a.x);
    const E* dy = static_cast<const E*>(a.dy);
    const WT* w = static_cast<const WT*>(a.weight);
    E* gx = static_cast<E*>(a.gx);
    float2* sums = static_cast<float2*>(ws);
    int n = back_groups(a.rows);
    float* part = reinterpret_cast<float*>(sums + a.rows);
    const bool ww = a.gweight, wb = a.gbias;
    if (vectors_fit<E>(a.width, 2048)) {
        const int nv = (int)(a.width / Vec<E>::W);
        auto go = [&](auto* kernel, int it, int at_once) {
            const int64_t want = (a.rows + at_once - 1) / at_once;
            n = (int)(want < kBackGrid ? want : kBackGrid);
            const int nt = ((nv + it - 1) / it + 31) / 32 * 32;
            kernel<<<n, nt, 0, st>>>(dy, x, w, a.mean, a.rstd, gx, part, a.rows, (int)a.width, ww, wb);
        };
        // the ring's size: two tensors' rows a stage; the column sums go over it at the end
        auto with_ring = [&](auto g, auto it) {
            constexpr int G = decltype(g)::value, IT = decltype(it)::value, NG = kRowWarps / G;
            const size_t bytes = (size_t)NG * kStages * 2 * a.width * sizeof(E) + (size_t)a.width * 4;
            const size_t sums = sizeof(float) * 32 * G * IT * Vec<E>::W;
            const size_t smem = bytes > sums ? bytes : sums;
            const int64_t want = (a.rows + NG - 1) / NG;
            n = (int)(want < kBackGrid ? want : kBackGrid);
            constexpr uint32_t most = 32 * G * IT * Vec<E>::W * (NG * kStages * 2 * sizeof(E) + 4);  // of the widest row
            const cudaError_t e = delta::allow<norm_back_ring<E, WT, IT, G>>(most);
            if (e == cudaSuccess)
                norm_back_ring<E, WT, IT, G><<<n, 32 * kRowWarps, smem, st>>>(dy, x, w, a.mean, a.rstd, gx, part, a.rows, (int)a.width, ww, wb,
                                                        status_word());
            return e;
        };
        auto by_vectors = [&](auto g) {
            const int it = (nv + 32 * decltype(g)::value - 1) / (32 * decltype(g)::value);
            if (it <= 1) return with_ring(g, std::integral_constant<int, 1>());
            if (it <= 2) return with_ring(g, std::integral_constant<int, 2>());
            return with_ring(g, std::integral_constant<int, 3>());
        };
        cudaError_t e = cudaSuccess;
        if (nv <= 96)
            e = by_vectors(std::integral_constant<int, 1>());
        else if (nv <= 192)
            e = by_vectors(std::integral_constant<int, 2>());
        else if (nv <= 384)
            e = by_vectors(std::integral_constant<int, 4>());
        else if (nv <= 768)
            e = by_vectors(std::integral_constant<int, 8>());
        else if (nv <= 1024)
            go(norm_back_rows<E, WT, 2, 2, 512>, 2, 2);
        else
            go(norm_back_rows<E, WT, 2, 1, 1024>, 2, 1);
        if (e != cudaSuccess) return e;
    } else {
        norm_back_sums<E, WT><<<(unsigned)(a.rows < 8192 ? a.rows : 8192), 256, 0, st>>>(dy, x, w, a.mean, a.rstd, sums,
                                                                                        a.rows, a.width);
        norm_back_cols<E, WT><<<dim3((unsigned)((a.width + 31) / 32), n), 256, 0, st>>>(
            dy, x, w, a.mean, a.rstd, sums, gx, part, a.rows, a.width, ww, wb);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!ww && !wb)) return e;
    // launched while the kernel before it runs, so that its CTAs are there when that ends
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.width + 31) / 32), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_back_join<WT>, static_cast<const float*>(part), n, a.width,
                              static_cast<WT*>(a.gweight), static_cast<WT*>(a.gbias));
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
