// The norm after a mixer, under its gate (the formulas stand at the head of blocknorm.cuh).

#pragma once

#include "blocknorm.cuh"

namespace cssd {
namespace {

// --------------------------------------------------------------- gated, forward
// TPR threads a group of a row, the group in registers as IT vectors a thread, and UN groups a team one after
// another in memory, all of whose loads come first; with at most a warp a group, no barrier.  Two groups a team:
// 16.9 us for 8192 x 1536 in groups of 64, one 19.1, four 17.4, eight 24.0.
template <typename E, typename W, int TPR, int IT, int UN>
__global__ void __launch_bounds__(TPR <= 32 ? 128 : TPR) gated_rows(GatedNormArgs a, int groups, unsigned units) {
    constexpr int V = Vec<E>::W, RPC = TPR <= 32 ? 128 / TPR : 1;
    __shared__ float red[32];
    const int tid = threadIdx.x % TPR, width = (int)a.group, nv = width / V;
    const unsigned u0 = blockIdx.x * (RPC * UN) + threadIdx.x / TPR;  // (unit n is u0 + n RPC)
    uint4 xr[UN][IT], zr[UN][IT];  // (as they come: half the registers of their values)
#pragma unroll
    for (int n = 0; n < UN; ++n) {
        const bool live = u0 + n * RPC < units;  // (with barriers a CTA has one group)
        const int64_t at = (int64_t)(u0 + n * RPC) * width;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (tid + TPR * i) * V;
            const bool in = live && c < width;
            xr[n][i] = in ? __ldcs(reinterpret_cast<const uint4*>(static_cast<const E*>(a.x) + at + c)) : make_uint4(0, 0, 0, 0);
            zr[n][i] = in ? __ldcs(reinterpret_cast<const uint4*>(static_cast<const E*>(a.z) + at + c)) : make_uint4(0, 0, 0, 0);
        }
    }
    const float inv = 1.f / (float)width;
#pragma unroll
    for (int n = 0; n < UN; ++n) {
        const unsigned unit = u0 + n * RPC;
        const bool live = unit < units;
        const int64_t at = (int64_t)unit * width;
        const int c0 = (int)(unit % (unsigned)groups) * width;
        float f[IT][V], z[IT][V];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            unpack<E>(xr[n][i], f[i]);
            unpack<E>(zr[n][i], z[i]);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                z[i][u] *= sigmoid<E>(z[i][u]);
                if (a.gate_first) f[i][u] *= z[i][u];
            }
        }
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
        if (!live) continue;
        if (tid == 0) {
            if (a.mean && a.layer) a.mean[unit] = m;
            if (a.rstd) a.rstd[unit] = r;
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (tid + TPR * i) * V;
            if (c >= width) break;
            float w[V], b[V];
            load_or<W, V>(static_cast<const W*>(a.weight), c0 + c, 1.f, w);
            load_or<W, V>(static_cast<const W*>(a.bias), c0 + c, 0.f, b);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                w[u] = fmaf((f[i][u] - m) * r, w[u], b[u]);
                if (!a.gate_first) w[u] *= z[i][u];
            }
            store<E, V>(static_cast<E*>(a.y) + at + c, w);
        }
    }
}

// Any width: a group is read again from the caches for each sum.
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
            return xv * (zv * sigmoid<E>(zv));
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
                v *= zv * sigmoid<E>(zv);
            }
            y[c] = from_f<E>(v);
        }
    }
}

// What a column needs of the gate: silu and its slope.
template <typename E>
__device__ __forceinline__ void gate_of(float z, float& gate, float& slope) {
    const float s = sigmoid<E>(z);
    gate = z * s;
    slope = s * fmaf(z, 1.f - s, 1.f);
}

// --------------------------------------------------------------- gradients, by a ring
// A ring row is a row of x and all its groups, where a group is 1, 2, 4 .. 32 whole vectors (`lanes` of a warp),
// or (lanes 0) one group of a row: a CTA then stays with the columns of group blockIdx.x % groups.
template <typename E, int IT, int G, bool FIRST>
__global__ void __launch_bounds__(32 * kRowWarps, 2) gated_back_ring(GatedNormArgs a, int lanes, float* __restrict__ part, unsigned* status) {
    constexpr int V = Vec<E>::W, NG = kRowWarps / G, TG = 32 * G;
    extern __shared__ __align__(128) unsigned char ring[];  // [group of warps][stage][x, z, dy], then the weights and biases
    __shared__ __align__(8) uint64_t full[NG][kStages];
    __shared__ float red[2][kRowWarps][2];
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, group = warp / G, gt = tid % TG;
    const int groups = (int)(a.width / a.group), mine_g = lanes ? 0 : (int)(blockIdx.x % groups), slices = lanes ? 1 : groups;
    const int width = (int)(lanes ? a.width : a.group), nv = width / V;
    const int64_t c0 = (int64_t)mine_g * width;
    const uint32_t eb = (uint32_t)width * sizeof(E), bytes = 3 * eb;
    delta::let_next_start();
    unsigned char* mine = ring + (size_t)group * kStages * bytes;
    float* sw = reinterpret_cast<float*>(ring + (size_t)NG * kStages * bytes);
    float* sb = sw + width;
    spread(sw, a.weight, a.wtype == CSSD_F32, a.xtype, 1.f, c0, width, tid, 32 * kRowWarps);
    spread(sb, a.bias, a.wtype == CSSD_F32, a.xtype, 0.f, c0, width, tid, 32 * kRowWarps);
    if (tid == 0) {
        s_gave_up = 0;
        for (int i = 0; i < NG; ++i)
            for (int j = 0; j < kStages; ++j) tc::mbar_init(&full[i][j], 1);
        tc::mbar_fence_init();
    }
    __syncthreads();
    float gw[IT][V], gb[IT][V];
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int u = 0; u < V; ++u) gw[i][u] = gb[i][u] = 0.f;
    const float inv = 1.f / (float)a.group;
    const int64_t step = (int64_t)(gridDim.x / slices) * NG, row0 = (int64_t)(blockIdx.x / slices) * NG + group;
    auto fetch = [&](int64_t k) {  // the k-th row of this group of warps
        const int64_t row = row0 + k * step, at = row * a.width + c0;
        if (row >= a.rows) return;
        uint64_t* bar = &full[group][k % kStages];
        const uint32_t to = tc::smem_u32(mine) + (uint32_t)(k % kStages) * bytes;
        tc::mbar_arrive_expect_tx(bar, bytes);
        tc::bulk_g2s(to, static_cast<const E*>(a.x) + at, eb, bar);
        tc::bulk_g2s(to + eb, static_cast<const E*>(a.z) + at, eb, bar);
        tc::bulk_g2s(to + 2 * eb, static_cast<const E*>(a.dy) + at, eb, bar);
    };
    if (gt == 0)
        for (int k = 0; k < kStages - 1; ++k) fetch(k);
    int64_t k = 0;
    for (int64_t row = row0; row < a.rows; row += step, ++k) {
        const int st = (int)(k % kStages);
        // (a wait that gives up: the row's results are wrong and the status word says so)
        float m[IT], r[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int v = gt + TG * i;
            const int64_t u = row * groups + (lanes ? (v < nv ? v / lanes : 0) : mine_g);
            m[i] = a.layer ? a.mean[u] : 0.f;
            r[i] = a.rstd[u];
        }
        if (!tc::mbar_wait_bounded(&full[group][st], (uint32_t)(k / kStages & 1), kNormWait)) s_gave_up = 1;
        const E* in = reinterpret_cast<const E*>(mine + (size_t)st * bytes);
        float s1[IT], s2[IT], sg[IT][V];  // (the sigmoids are kept from one pass to the next)
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int v = gt + TG * i;
            s1[i] = s2[i] = 0.f;
            if (v < nv) {
                float x[V], z[V], d[V], w[V];
                load<E, V>(in + v * V, x);
                load<E, V>(in + width + v * V, z);
                load<E, V>(in + 2 * width + v * V, d);
                load<float, V>(sw + v * V, w);
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    sg[i][u] = sigmoid<E>(z[u]);
                    const float gate = z[u] * sg[i][u];
                    const float hh = ((FIRST ? x[u] * gate : x[u]) - m[i]) * r[i], du = FIRST ? d[u] : d[u] * gate, g = du * w[u];
                    s1[i] += g;
                    s2[i] = fmaf(g, hh, s2[i]);
                    gw[i][u] = fmaf(du, hh, gw[i][u]);
                    gb[i][u] += du;
                }
            }
        }
        if (lanes) {
#pragma unroll
            for (int i = 0; i < IT; ++i)
                for (int o = lanes / 2; o; o >>= 1) {
                    s1[i] += __shfl_xor_sync(0xffffffffu, s1[i], o);
                    s2[i] += __shfl_xor_sync(0xffffffffu, s2[i], o);
                }
            group_barrier<G>(group);
        } else {
            float p = 0.f, q = 0.f;
#pragma unroll
            for (int i = 0; i < IT; ++i) p += s1[i], q += s2[i];
            const float2 sum = group_sums<G>(p, q, red[k & 1], group, warp, lane);
#pragma unroll
            for (int i = 0; i < IT; ++i) s1[i] = sum.x, s2[i] = sum.y;
        }
        // every thread of the group is past the row before: its stage is free
        if (gt == 0) fetch(k + kStages - 1);
        const int64_t at = row * a.width + c0;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int v = gt + TG * i;
            if (v < nv) {
                const float t1 = a.layer ? s1[i] * inv : 0.f, t2 = s2[i] * inv;
                float x[V], z[V], d[V], w[V], b[V];
                load<E, V>(in + v * V, x);
                load<E, V>(in + width + v * V, z);
                load<E, V>(in + 2 * width + v * V, d);
                load<float, V>(sw + v * V, w);
                if (!FIRST) load<float, V>(sb + v * V, b);
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    const float gate = z[u] * sg[i][u], slope = sg[i][u] * fmaf(z[u], 1.f - sg[i][u], 1.f);
                    const float hh = ((FIRST ? x[u] * gate : x[u]) - m[i]) * r[i], du = FIRST ? d[u] : d[u] * gate;
                    const float dh = r[i] * (du * w[u] - t1 - hh * t2);
                    z[u] = (FIRST ? dh * x[u] : d[u] * fmaf(hh, w[u], b[u])) * slope;
                    x[u] = FIRST ? dh * gate : dh;
                }
                store<E, V>(static_cast<E*>(a.gx) + at + v * V, x);
                store<E, V>(static_cast<E*>(a.gz) + at + v * V, z);
            }
        }
    }
    if (gt == 0 && s_gave_up)  // no copy may land in shared memory that is no longer this CTA's
        for (int64_t e = k > kStages ? k - kStages : 0; e < k; ++e)
            tc::mbar_wait_bounded(&full[group][e % kStages], (uint32_t)(e / kStages & 1), kNormWait);
    // the groups' column sums, one after another (the copies have all been waited for)
    __syncthreads();
    float* sum = reinterpret_cast<float*>(ring);
    float* to = part + (int64_t)(blockIdx.x / slices) * 2 * a.width + c0;
    join_groups<V, IT, G>(gw, sum, to, a.gweight, width, group, gt, tid);
    join_groups<V, IT, G>(gb, sum, to + a.width, a.gbias, width, group, gt, tid);
    if (tid == 0 && s_gave_up && status) atomicOr(status, kStatusNorm);
}

// --------------------------------------------------------------- gradients, streamed
// First the two means of every group, then dx and the column sums.
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
            gate_of<E>(to_f(static_cast<const E*>(a.z)[at + c]), gate, slope);
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
            gate_of<E>(to_f(z[i]), gate, slope);
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

template <typename E, typename W>
cudaError_t gated_fwd(const GatedNormArgs& a, cudaStream_t st) {
    const int64_t units = a.rows * (a.width / a.group);
    if (vectors_fit<E>(a.group, 1024))
        return by_vectors<true>(a.group / Vec<E>::W, [&](auto t, auto i) {
            constexpr int TPR = decltype(t)::value, IT = decltype(i)::value, RPC = TPR <= 32 ? 128 / TPR : 1;
            constexpr int MANY = TPR > 32 || IT > 2 ? 1 : 2 / IT;
            auto go = [&](auto un) {
                constexpr int UN = decltype(un)::value;
                gated_rows<E, W, TPR, IT, UN><<<(unsigned)((units + RPC * UN - 1) / (RPC * UN)), TPR * RPC, 0, st>>>(
                    a, (int)(a.width / a.group), (unsigned)units);
                return cudaGetLastError();
            };
            // (few groups: one a team, so that they spread over the SMs)
            if constexpr (MANY > 1)
                if (units >= (int64_t)RPC * MANY * 152) return go(std::integral_constant<int, MANY>());
            return go(std::integral_constant<int, 1>());
        });
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
    int n = back_groups(a.rows);
    constexpr int V = Vec<E>::W;
    const int64_t gv = a.group / V, groups = a.width / a.group;
    RingPlan plan;
    bool ring = false;
    int lanes = 0;
    if (a.group % V == 0 && groups > 1 && gv <= 32 && (gv & (gv - 1)) == 0) {
        lanes = (int)gv;
        ring = plan_ring(a.width / V, V, (size_t)3 * a.width * sizeof(E), (size_t)8 * a.width, plan);
    }
    // (a warp a group at least: narrow ones are streamed.  8192 x 2040, us, ring and streamed: groups of 3 vectors 393 and
    // 200, of 5 261 and 185, of 6 234 and 171 but 31 and 49 for 1000 rows, of 10 158 and 143 (29 and 43), of 20 69 and 126)
    if (!ring && a.group % V == 0 && groups <= kBackGrid && gv >= 6) {
        lanes = 0;
        ring = plan_ring(gv, V, (size_t)3 * a.group * sizeof(E), (size_t)8 * a.group, plan);
    }
    if (ring) {
        const cudaError_t e = by_plan(plan, [&](auto g, auto i) {
            constexpr int G = decltype(g)::value, IT = decltype(i)::value;
            // CTAs a group: what fills the SMs, and with many groups so many that a thread adds up 64 rows in fp32
            // (as many as the partial sums have room for; 20000 rows of 304 groups, one CTA each: 620 2^-24 off)
            const int64_t slices = lanes ? 1 : groups, NG = kRowWarps / G, want = (a.rows + NG - 1) / NG;
            const int64_t fill = kBackGrid / slices, few = grid_of((a.rows + 64 * NG - 1) / (64 * NG), kBackGrid);
            n = (int)grid_of(want, fill > few ? fill : few);
            auto go = [&](auto first) {
                constexpr bool FIRST = decltype(first)::value;
                const cudaError_t e = delta::allow<gated_back_ring<E, IT, G, FIRST>>(220 << 10);
                if (e == cudaSuccess)
                    gated_back_ring<E, IT, G, FIRST><<<(unsigned)(n * slices), 32 * kRowWarps, plan.smem, st>>>(a, lanes, part, status_word());
                return e == cudaSuccess ? cudaGetLastError() : e;
            };
            return a.gate_first ? go(std::true_type()) : go(std::false_type());
        });
        if (e != cudaSuccess) return e;
        return join<W>(part, n, a.width, 2, static_cast<W*>(a.gweight), static_cast<W*>(a.gbias), static_cast<W*>(nullptr), st);
    }
    if (a.group <= 1024)
        gated_back_sums<E, W, 32><<<grid_of((units + 7) / 8, 8192), 256, 0, st>>>(a, sums);
    else
        gated_back_sums<E, W, 256><<<grid_of(units, 8192), 256, 0, st>>>(a, sums);
    gated_back_cols<E, W><<<dim3((unsigned)((a.width + 31) / 32), n), 256, 0, st>>>(a, sums, part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return join<W>(part, n, a.width, 2, static_cast<W*>(a.gweight), static_cast<W*>(a.gbias), static_cast<W*>(nullptr), st);
}

template <typename E>
cudaError_t gated_forward(const GatedNormArgs& a, cudaStream_t st) {
    return or_float(a.wtype == CSSD_F32, static_cast<E*>(nullptr), [&](auto* w) { return gated_fwd<E, To<decltype(w)>>(a, st); });
}
template <typename E>
cudaError_t gated_backward(const GatedNormArgs& a, void* ws, cudaStream_t st) {
    return or_float(a.wtype == CSSD_F32, static_cast<E*>(nullptr), [&](auto* w) { return gated_bwd<E, To<decltype(w)>>(a, ws, st); });
}

}  // namespace
}  // namespace cssd
