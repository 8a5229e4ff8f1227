// One token of linear attention with a decay for each head, for every (batch
// row, value head):
//     S = e^g S + k v^T,   o = scale S^T q
// The state passes through the registers once: bound by its bytes, read and
// written once (2 x 4 N P a head).
//
// A CTA owns 32 state columns of one head (they never mix), so that a decode
// batch has several CTAs a head to spread over the SMs and a single sequence
// still gets P / 32 of them a head.  Eight lanes hold a row's 32 columns as
// float4 (128 contiguous bytes), 16 row groups of them N / 16 rows each.
// e^g is two floats (exp_pair): its error is the same for every token that a head with one decay remembers.
// Measured: 256 rows of a pool of 288, 32 heads, 128/64: 82 us on the device, 6.7 TB/s (98 % of the copy rate), 83 a call
// among others; one row of 12 heads, 64/64: 2 us, 15 a call from Python.

#include "cssd_internal.h"
#include "linattn_common.cuh"

namespace cssd {
namespace linattn {
namespace {

constexpr int SPW = 32, SNT = 128, SRG = SNT / 8;

template <typename E, int RPT>
__global__ void __launch_bounds__(SNT) step_kernel(float* __restrict__ h, const int* __restrict__ slots, int64_t nslots,
                                                   const E* __restrict__ q, const E* __restrict__ k,
                                                   const E* __restrict__ v, const float* __restrict__ g, bool g_tokens,
                                                   float scale, E* __restrict__ o, int H, int G, int P) {
    constexpr int N = RPT * SRG;
    __shared__ float sk[N], sq[N];
    __shared__ float4 part[SNT / 32][8];
    const int np = (P + SPW - 1) / SPW;
    const int bh = (int)(blockIdx.x / np), p = (int)(blockIdx.x % np) * SPW + 4 * (threadIdx.x % 8);
    const int b = bh / H, hd = bh - b * H, KH = H / G;
    const int tid = threadIdx.x, rg = tid / 8, lane = tid % 32, warp = tid / 32;
    const int64_t slot = slots ? (int64_t)slots[b] : (int64_t)b;
    E* orow = o + (int64_t)bh * P;
    if (slot < 0 || slot >= nslots) {  // no state: the row's output is zero
        if (tid < 8 && p < P)
#pragma unroll
            for (int u = 0; u < 4; ++u) orow[p + u] = from_f<E>(0.f);
        return;
    }
    float4* hs = reinterpret_cast<float4*>(h + ((slot * H + hd) * N) * (int64_t)P + p);
    const int64_t rs = P / 4;
    const bool live = p < P;
    float4 s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) s[i] = live ? __ldcs(hs + (rg + SRG * i) * rs) : make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t ko = ((int64_t)b * KH + hd / G) * N;
    for (int n = tid; n < N; n += SNT) {
        sk[n] = to_f(k[ko + n]);
        sq[n] = to_f(q[ko + n]);
    }
    const float2 a = exp_pair({g[g_tokens ? bh : hd], 0.f});
    float4 vv = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
        const E* vr = v + (int64_t)bh * P + p;
        vv = make_float4(to_f(vr[0]), to_f(vr[1]), to_f(vr[2]), to_f(vr[3]));
    }
    __syncthreads();
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float kn = sk[rg + SRG * i], qn = sq[rg + SRG * i];
        s[i].x = fmaf(a.x, s[i].x, fmaf(a.y, s[i].x, kn * vv.x)), s[i].y = fmaf(a.x, s[i].y, fmaf(a.y, s[i].y, kn * vv.y));
        s[i].z = fmaf(a.x, s[i].z, fmaf(a.y, s[i].z, kn * vv.z)), s[i].w = fmaf(a.x, s[i].w, fmaf(a.y, s[i].w, kn * vv.w));
        r.x = fmaf(s[i].x, qn, r.x), r.y = fmaf(s[i].y, qn, r.y);
        r.z = fmaf(s[i].z, qn, r.z), r.w = fmaf(s[i].w, qn, r.w);
        if (live) __stcs(hs + (rg + SRG * i) * rs, s[i]);
    }
#pragma unroll
    for (int w = 8; w <= 16; w <<= 1) {  // over the warp's four row groups
        r.x += __shfl_xor_sync(0xffffffffu, r.x, w), r.y += __shfl_xor_sync(0xffffffffu, r.y, w);
        r.z += __shfl_xor_sync(0xffffffffu, r.z, w), r.w += __shfl_xor_sync(0xffffffffu, r.w, w);
    }
    if (lane < 8) part[warp][lane] = r;
    __syncthreads();
    if (tid < 8 && live) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < SNT / 32; ++w) {
            const float4 x = part[w][tid];
            t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
        }
        orow[p] = from_f<E>(scale * t.x);
        orow[p + 1] = from_f<E>(scale * t.y);
        orow[p + 2] = from_f<E>(scale * t.z);
        orow[p + 3] = from_f<E>(scale * t.w);
    }
}

template <typename E>
cudaError_t step(const LinattnStepArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.P + SPW - 1) / SPW * a.Bz * a.H);
    auto go = [&](auto* kernel) {
        kernel<<<grid, SNT, 0, st>>>(a.h, a.slots, a.nslots, static_cast<const E*>(a.q), static_cast<const E*>(a.k),
                                     static_cast<const E*>(a.v), a.g, a.g_tokens, a.scale, static_cast<E*>(a.o), (int)a.H,
                                     (int)(a.H / a.KH), (int)a.P);
        return cudaGetLastError();
    };
    switch (a.N / SRG) {
        case 1: return go(step_kernel<E, 1>);
        case 2: return go(step_kernel<E, 2>);
        case 3: return go(step_kernel<E, 3>);
        case 4: return go(step_kernel<E, 4>);
        case 5: return go(step_kernel<E, 5>);
        case 6: return go(step_kernel<E, 6>);
        case 7: return go(step_kernel<E, 7>);
        case 8: return go(step_kernel<E, 8>);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace linattn

cudaError_t launch_linattn_step(const LinattnStepArgs& a, cudaStream_t st) {
    if (a.dtype == CSSD_BF16) return linattn::step<__nv_bfloat16>(a, st);
    if (a.dtype == CSSD_F16) return linattn::step<__half>(a, st);
    return linattn::step<float>(a, st);
}

}  // namespace cssd
