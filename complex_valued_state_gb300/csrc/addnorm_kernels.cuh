// The norm before a block, with the residual sum and its scale (the formulas stand at the head of blocknorm.cuh).

#pragma once

#include "blocknorm.cuh"

namespace cssd {
namespace {

// --------------------------------------------------------------- add, forward
// residual + alpha x, the product rounded before the sum: with a decimal alpha (0.7) of tensors of few bits the sum is
// often a tie of the result's type, which the product's rounding restores and alpha's own error would break (6 of
// 10000 elements of bfloat16 sums went the other way in one operation).
__device__ __forceinline__ float scaled_sum(float residual, float alpha, float x) { return __fadd_rn(residual, __fmul_rn(alpha, x)); }

// TPR threads a row, the row in registers as IT vectors a thread; with at most a warp a row, no barrier.
template <typename E, typename R, typename W, int TPR, int IT>
__global__ void __launch_bounds__(TPR <= 32 ? 128 : TPR) add_rows(AddNormArgs a) {
    constexpr int V = Vec<E>::W, RPC = TPR <= 32 ? 128 / TPR : 1;
    __shared__ float red[32];
    const int tid = threadIdx.x % TPR, width = (int)a.width, nv = width / V;
    const int64_t row = (int64_t)blockIdx.x * RPC + threadIdx.x / TPR;
    const bool live = row < a.rows;  // (with barriers a CTA has one row)
    const int64_t at = (live ? row : 0) * width;
    const E* x = static_cast<const E*>(a.x) + at;
    const R* res = static_cast<const R*>(a.residual) + at;
    R* s = static_cast<R*>(a.s) + at;
    float f[IT][V];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (tid + TPR * i) * V;
#pragma unroll
        for (int u = 0; u < V; ++u) f[i][u] = 0.f;
        if (live && c < width) {
            float xv[V];
            load_once<R, V>(res + c, f[i]);
            load_once<E, V>(x + c, xv);
            if (a.scale) {
                float sc[V];
                load<W, V>(static_cast<const W*>(a.scale) + c, sc);
#pragma unroll
                for (int u = 0; u < V; ++u) xv[u] *= sc[u];
            }
#pragma unroll
            for (int u = 0; u < V; ++u) f[i][u] = to_f(from_f<R>(scaled_sum(f[i][u], a.alpha, xv[u])));
        }
    }
    const float inv = 1.f / (float)width;
    float m = 0.f, t = 0.f;
    if (a.layer) {
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int u = 0; u < V; ++u) t += f[i][u];
        m = lanes_sum<TPR>(t, red, tid) * inv;
        t = 0.f;
    }
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if (tid + TPR * i < nv)
#pragma unroll
            for (int u = 0; u < V; ++u) t = fmaf(f[i][u] - m, f[i][u] - m, t);
    const float r = rsqrtf(lanes_sum<TPR>(t, red, tid) * inv + a.eps);
    if (!live) return;
    if (tid == 0) {
        if (a.mean && a.layer) a.mean[row] = m;
        if (a.rstd) a.rstd[row] = r;
    }
    E* y = static_cast<E*>(a.y) + at;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (tid + TPR * i) * V;
        if (c >= width) break;
        float w[V], b[V];
        store<R, V>(s + c, f[i]);
        load_or<W, V>(static_cast<const W*>(a.weight), c, 1.f, w);
        load_or<W, V>(static_cast<const W*>(a.bias), c, 0.f, b);
#pragma unroll
        for (int u = 0; u < V; ++u) w[u] = fmaf((f[i][u] - m) * r, w[u], b[u]);
        store<E, V>(y + c, w);
    }
}

// Any width: the row is read again from the caches for each sum.
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
            s[c] = from_f<R>(scaled_sum(to_f(res[c]), a.alpha, at_or(sc, c, 1.f) * to_f(x[c])));
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

// --------------------------------------------------------------- gradients, by a ring
template <typename E, typename R, int IT, int G>
__global__ void __launch_bounds__(32 * kRowWarps, 2) add_back_ring(AddNormArgs a, float* __restrict__ part, unsigned* status) {
    constexpr int V = Vec<E>::W, NG = kRowWarps / G, TG = 32 * G;
    extern __shared__ __align__(128) unsigned char ring[];  // [group][stage][s, ds, dy, x], then the weights and scales
    __shared__ __align__(8) uint64_t full[NG][kStages];
    __shared__ float red[2][kRowWarps][2];
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, group = warp / G, gt = tid % TG;
    const int width = (int)a.width, nv = width / V;
    const uint32_t rb = (uint32_t)width * sizeof(R), eb = (uint32_t)width * sizeof(E);
    const bool has_ds = a.ds, has_x = a.gscale;
    const uint32_t at_ds = rb, at_dy = rb * (1 + has_ds), at_x = at_dy + eb, bytes = at_x + (has_x ? eb : 0);
    delta::let_next_start();
    unsigned char* mine = ring + (size_t)group * kStages * bytes;
    float* sw = reinterpret_cast<float*>(ring + (size_t)NG * kStages * bytes);
    float* ss = sw + width;  // alpha scale
    spread(sw, a.weight, a.wtype == CSSD_F32, a.xtype, 1.f, 0, width, tid, 32 * kRowWarps);
    spread(ss, a.scale, a.wtype == CSSD_F32, a.xtype, 1.f, 0, width, tid, 32 * kRowWarps);
    if (tid == 0) {
        s_gave_up = 0;
        for (int i = 0; i < NG; ++i)
            for (int j = 0; j < kStages; ++j) tc::mbar_init(&full[i][j], 1);
        tc::mbar_fence_init();
    }
    __syncthreads();
    float gs[IT][V], gw[IT][V], gb[IT][V];
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int u = 0; u < V; ++u) gs[i][u] = gw[i][u] = gb[i][u] = 0.f;
    const float inv = 1.f / (float)width;
    const int64_t step = (int64_t)gridDim.x * NG, row0 = (int64_t)blockIdx.x * NG + group;
    auto fetch = [&](int64_t k) {  // the group's k-th row
        const int64_t row = row0 + k * step;
        if (row >= a.rows) return;
        uint64_t* bar = &full[group][k % kStages];
        const uint32_t to = tc::smem_u32(mine) + (uint32_t)(k % kStages) * bytes;
        tc::mbar_arrive_expect_tx(bar, bytes);
        tc::bulk_g2s(to, static_cast<const R*>(a.s) + row * width, rb, bar);
        if (has_ds) tc::bulk_g2s(to + at_ds, static_cast<const R*>(a.ds) + row * width, rb, bar);
        tc::bulk_g2s(to + at_dy, static_cast<const E*>(a.dy) + row * width, eb, bar);
        if (has_x) tc::bulk_g2s(to + at_x, static_cast<const E*>(a.x) + row * width, eb, bar);
    };
    if (gt == 0)
        for (int k = 0; k < kStages - 1; ++k) fetch(k);
    int64_t k = 0;
    for (int64_t row = row0; row < a.rows; row += step, ++k) {
        const int st = (int)(k % kStages);
        const float m = a.layer ? a.mean[row] : 0.f, r = a.rstd[row];
        // (a wait that gives up: the row's results are wrong and the status word says so)
        if (!tc::mbar_wait_bounded(&full[group][st], (uint32_t)(k / kStages & 1), kNormWait)) s_gave_up = 1;
        const unsigned char* in = mine + (size_t)st * bytes;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int v = gt + TG * i;
            if (v < nv) {
                float h[V], d[V], w[V];
                load<R, V>(reinterpret_cast<const R*>(in) + v * V, h);
                load<E, V>(reinterpret_cast<const E*>(in + at_dy) + v * V, d);
                load<float, V>(sw + v * V, w);
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    const float hh = (h[u] - m) * r, g = d[u] * w[u];
                    s1 += g;
                    s2 = fmaf(g, hh, s2);
                    gw[i][u] = fmaf(d[u], hh, gw[i][u]);
                    gb[i][u] += d[u];
                }
            }
        }
        const float2 sum = group_sums<G>(s1, s2, red[k & 1], group, warp, lane);
        // every thread of the group is past the row before: its stage is free
        if (gt == 0) fetch(k + kStages - 1);
        const float t1 = a.layer ? sum.x * inv : 0.f, t2 = sum.y * inv;
        R* gr = static_cast<R*>(a.gresidual) + row * width;
        E* gx = static_cast<E*>(a.gx) + row * width;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int v = gt + TG * i;
            if (v < nv) {
                float h[V], d[V], w[V], e[V];
                load<R, V>(reinterpret_cast<const R*>(in) + v * V, h);
                load<E, V>(reinterpret_cast<const E*>(in + at_dy) + v * V, d);
                load<float, V>(sw + v * V, w);
                if (has_ds)
                    load<R, V>(reinterpret_cast<const R*>(in + at_ds) + v * V, e);
                else
#pragma unroll
                    for (int u = 0; u < V; ++u) e[u] = 0.f;
#pragma unroll
                for (int u = 0; u < V; ++u) h[u] = fmaf(r, d[u] * w[u] - t1 - (h[u] - m) * r * t2, e[u]);
                store<R, V>(gr + v * V, h);
                if (has_x) {
                    load<E, V>(reinterpret_cast<const E*>(in + at_x) + v * V, e);
#pragma unroll
                    for (int u = 0; u < V; ++u) gs[i][u] = fmaf(h[u], e[u], gs[i][u]);
                }
                load<float, V>(ss + v * V, e);
#pragma unroll
                for (int u = 0; u < V; ++u) h[u] *= a.alpha * e[u];
                store<E, V>(gx + v * V, h);
            }
        }
    }
    if (gt == 0 && s_gave_up)  // no copy may land in shared memory that is no longer this CTA's
        for (int64_t e = k > kStages ? k - kStages : 0; e < k; ++e)
            tc::mbar_wait_bounded(&full[group][e % kStages], (uint32_t)(e / kStages & 1), kNormWait);
    // the groups' column sums, one after another (the copies have all been waited for)
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int u = 0; u < V; ++u) gs[i][u] *= a.alpha;
    float* sum = reinterpret_cast<float*>(ring);
    float* to = part + (int64_t)blockIdx.x * 3 * width;
    join_groups<V, IT, G>(gs, sum, to, a.gscale, width, group, gt, tid);
    join_groups<V, IT, G>(gw, sum, to + width, a.gweight, width, group, gt, tid);
    join_groups<V, IT, G>(gb, sum, to + 2 * width, a.gbias, width, group, gt, tid);
    if (tid == 0 && s_gave_up && status) atomicOr(status, kStatusNorm);
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

template <typename E, typename R, typename W>
cudaError_t add_fwd(const AddNormArgs& a, cudaStream_t st) {
    if (vectors_fit<E>(a.width, 4096))
        return by_vectors<false>(a.width / Vec<E>::W, [&](auto t, auto i) {
            constexpr int TPR = decltype(t)::value, IT = decltype(i)::value, RPC = TPR <= 32 ? 128 / TPR : 1;
            add_rows<E, R, W, TPR, IT><<<(unsigned)((a.rows + RPC - 1) / RPC), TPR * RPC, 0, st>>>(a);
            return cudaGetLastError();
        });
    add_stream<E, R, W><<<grid_of(a.rows, 8192), 256, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename E, typename R, typename W>
cudaError_t add_bwd(const AddNormArgs& a, void* ws, cudaStream_t st) {
    float2* sums = static_cast<float2*>(ws);
    float* part = reinterpret_cast<float*>(sums + a.rows);
    int n = back_groups(a.rows);
    RingPlan plan;
    const size_t w = (size_t)a.width;
    if (vectors_fit<E>(a.width, 4096) &&
        plan_ring(a.width / Vec<E>::W, Vec<E>::W, w * ((a.ds ? 2 : 1) * sizeof(R) + (a.gscale ? 2 : 1) * sizeof(E)), 8 * w, plan)) {
        const cudaError_t e = by_plan(plan, [&](auto g, auto i) {
            constexpr int G = decltype(g)::value, IT = decltype(i)::value;
            const int64_t want = (a.rows + kRowWarps / G - 1) / (kRowWarps / G);
            n = (int)(want < kBackGrid ? want : kBackGrid);
            const cudaError_t e = delta::allow<add_back_ring<E, R, IT, G>>(220 << 10);
            if (e == cudaSuccess) add_back_ring<E, R, IT, G><<<n, 32 * kRowWarps, plan.smem, st>>>(a, part, status_word());
            return e == cudaSuccess ? cudaGetLastError() : e;
        });
        if (e != cudaSuccess) return e;
        return join<W>(part, n, a.width, 3, static_cast<W*>(a.gscale), static_cast<W*>(a.gweight), static_cast<W*>(a.gbias), st);
    }
    add_back_sums<E, R, W><<<grid_of(a.rows, 8192), 256, 0, st>>>(a, sums);
    add_back_cols<E, R, W><<<dim3((unsigned)((a.width + 31) / 32), n), 256, 0, st>>>(a, sums, part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return join<W>(part, n, a.width, 3, static_cast<W*>(a.gscale), static_cast<W*>(a.gweight), static_cast<W*>(a.gbias), st);
}

template <typename E, typename F>
cudaError_t add_types(const AddNormArgs& a, F f) {
    E* e = nullptr;
    return or_float(a.rtype == CSSD_F32, e, [&](auto* r) { return or_float(a.wtype == CSSD_F32, e, [&](auto* w) { return f(r, w); }); });
}
template <typename E>
cudaError_t add_forward(const AddNormArgs& a, cudaStream_t st) {
    return add_types<E>(a, [&](auto* r, auto* w) { return add_fwd<E, To<decltype(r)>, To<decltype(w)>>(a, st); });
}
template <typename E>
cudaError_t add_backward(const AddNormArgs& a, void* ws, cudaStream_t st) {
    return add_types<E>(a, [&](auto* r, auto* w) { return add_bwd<E, To<decltype(r)>, To<decltype(w)>>(a, ws, st); });
}

}  // namespace
}  // namespace cssd
