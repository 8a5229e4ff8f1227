// One token of the gated delta rule for every (batch row, value head):
//     S' = e^g S,  p = S'^T k,  r = S'^T q,  e = beta (v - p)
//     S  = S' + k e^T,          o = scale (r + (k.q) e)
// Both inner products with the state are taken from the state as it was read,
// so it passes through the registers once: bound by the state's bytes, read
// and written once (2 x 4 N P per head).
//
// A CTA owns PW = 32 state columns of one head (they never mix), so a decode
// batch has several CTAs a head to spread over the SMs and a single sequence
// still gets N P / 4096 of them a head.  Eight lanes hold a row's 32 columns
// as float4 (128 contiguous bytes), 16 row groups of them N / 16 rows each.
// Measured: 256 x 32 heads, 128/64: 81 us, 6.7 TB/s; 77 rows of a pool, 32
// heads, 128/128: 50 us, 6.4 TB/s; one row of 12 heads, 64/64: 2.2 us.

#include "cssd_internal.h"
#include "delta_common.cuh"

namespace cssd {
namespace delta {
namespace {

constexpr int SPW = 32, SNT = 128, SRG = SNT / 8;

template <typename E, int RPT>
__global__ void __launch_bounds__(SNT) delta_step_kernel(float* __restrict__ h, const int* __restrict__ slots,
                                                         int64_t nslots, const E* __restrict__ q,
                                                         const E* __restrict__ k, const E* __restrict__ v,
                                                         const float* __restrict__ g, const float* __restrict__ beta,
                                                         float scale, E* __restrict__ o, int H, int G, int P) {
    constexpr int N = RPT * SRG;
    __shared__ float sk[N], sq[N], s_kq[SNT / 32];
    __shared__ float4 part[2][SNT / 32][8];
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
    float kq = 0.f;
    for (int n = tid; n < N; n += SNT) {
        sk[n] = to_f(k[ko + n]);
        sq[n] = to_f(q[ko + n]);
        kq = fmaf(sk[n], sq[n], kq);
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, w);
    if (lane == 0) s_kq[warp] = kq;
    const float a = expf(g[bh]), bt = beta[bh];
    float4 vv = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
        const E* vr = v + (int64_t)bh * P + p;
        vv = make_float4(to_f(vr[0]), to_f(vr[1]), to_f(vr[2]), to_f(vr[3]));
    }
    __syncthreads();
    float4 dp = make_float4(0.f, 0.f, 0.f, 0.f), dr = dp;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float kn = sk[rg + SRG * i], qn = sq[rg + SRG * i];
        s[i].x *= a, s[i].y *= a, s[i].z *= a, s[i].w *= a;
        dp.x = fmaf(s[i].x, kn, dp.x), dp.y = fmaf(s[i].y, kn, dp.y);
        dp.z = fmaf(s[i].z, kn, dp.z), dp.w = fmaf(s[i].w, kn, dp.w);
        dr.x = fmaf(s[i].x, qn, dr.x), dr.y = fmaf(s[i].y, qn, dr.y);
        dr.z = fmaf(s[i].z, qn, dr.z), dr.w = fmaf(s[i].w, qn, dr.w);
    }
#pragma unroll
    for (int w = 8; w <= 16; w <<= 1) {  // over the warp's four row groups
        dp.x += __shfl_xor_sync(0xffffffffu, dp.x, w), dp.y += __shfl_xor_sync(0xffffffffu, dp.y, w);
        dp.z += __shfl_xor_sync(0xffffffffu, dp.z, w), dp.w += __shfl_xor_sync(0xffffffffu, dp.w, w);
        dr.x += __shfl_xor_sync(0xffffffffu, dr.x, w), dr.y += __shfl_xor_sync(0xffffffffu, dr.y, w);
        dr.z += __shfl_xor_sync(0xffffffffu, dr.z, w), dr.w += __shfl_xor_sync(0xffffffffu, dr.w, w);
    }
    if (lane < 8) {
        part[0][warp][lane] = dp;
        part[1][warp][lane] = dr;
    }
    __syncthreads();
    dp = dr = make_float4(0.f, 0.f, 0.f, 0.f);
    kq = 0.f;
#pragma unroll
    for (int w = 0; w < SNT / 32; ++w) {
        const float4 x = part[0][w][tid % 8], y = part[1][w][tid % 8];
        dp.x += x.x, dp.y += x.y, dp.z += x.z, dp.w += x.w;
        dr.x += y.x, dr.y += y.y, dr.z += y.z, dr.w += y.w;
        kq += s_kq[w];
    }
    const float4 e = make_float4(bt * (vv.x - dp.x), bt * (vv.y - dp.y), bt * (vv.z - dp.z), bt * (vv.w - dp.w));
    if (!live) return;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float kn = sk[rg + SRG * i];
        s[i].x = fmaf(kn, e.x, s[i].x), s[i].y = fmaf(kn, e.y, s[i].y);
        s[i].z = fmaf(kn, e.z, s[i].z), s[i].w = fmaf(kn, e.w, s[i].w);
        __stcs(hs + (rg + SRG * i) * rs, s[i]);
    }
    if (tid < 8) {
        orow[p] = from_f<E>(scale * fmaf(kq, e.x, dr.x));
        orow[p + 1] = from_f<E>(scale * fmaf(kq, e.y, dr.y));
        orow[p + 2] = from_f<E>(scale * fmaf(kq, e.z, dr.z));
        orow[p + 3] = from_f<E>(scale * fmaf(kq, e.w, dr.w));
    }
}

template <typename E>
cudaError_t step(const DeltaStepArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.P + SPW - 1) / SPW * a.Bz * a.H);
    auto go = [&](auto* kernel) {
        kernel<<<grid, SNT, 0, st>>>(a.h, a.slots, a.nslots, static_cast<const E*>(a.q), static_cast<const E*>(a.k),
                                     static_cast<const E*>(a.v), a.g, a.beta, a.scale, static_cast<E*>(a.o), (int)a.H,
                                     (int)(a.H / a.KH), (int)a.P);
        return cudaGetLastError();
    };
    switch (a.N / SRG) {
        case 1: return go(delta_step_kernel<E, 1>);
        case 2: return go(delta_step_kernel<E, 2>);
        case 3: return go(delta_step_kernel<E, 3>);
        case 4: return go(delta_step_kernel<E, 4>);
        case 5: return go(delta_step_kernel<E, 5>);
        case 6: return go(delta_step_kernel<E, 6>);
        case 7: return go(delta_step_kernel<E, 7>);
        case 8: return go(delta_step_kernel<E, 8>);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace delta

cudaError_t launch_delta_step(const DeltaStepArgs& a, cudaStream_t st) {
    if (a.dtype == CSSD_BF16) return delta::step<__nv_bfloat16>(a, st);
    if (a.dtype == CSSD_F16) return delta::step<__half>(a, st);
    return delta::step<float>(a, st);
}

}  // namespace cssd
