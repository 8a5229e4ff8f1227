// Linear attention with a decay for each head, over a sequence:
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// in chunks of C tokens.  With G_i the running sum of g in a chunk and
// M_ij = e^{G_i - G_j} (i >= j),
//     o_i   = scale (e^{G_i} q_i S + sum_j M_ij (q_i.k_j) v_j)
//     S+    = e^{G_end} S + sum_j e^{G_end - G_j} k_j v_j^T
// and, dS+ being the gradient of the state that leaves the chunk,
//     dq_i  = scale (e^{G_i} do_i S^T + sum_j M_ij (do_i.v_j) k_j)
//     dk_j  = e^{G_end - G_j} v_j dS+^T + scale sum_i M_ij (do_i.v_j) q_i
//     dv_j  = e^{G_end - G_j} k_j dS+   + scale sum_i M_ij (q_i.k_j) do_i
//     dS    = e^{G_end} dS+ + sum_i scale e^{G_i} q_i do_i^T
//     dg_t  = e^{G_end} <S, dS+> + sum_{all j} c_j + sum_{u >= t} (q_u.dq_u - k_u.dk_u)
// with c_j the first term's share of k_j.dk_j.  (dg_t = <e^{g_t} S_{t-1}, dL/dS_t>; what leaves the chunk
// is <S+, dS+>, the terms before the last sum.)
//
// Three kernels:
//   states   walks the chunks of a row and head (or of a segment of them) and
//            leaves the state before each chunk; for the gradients the same walk
//            backwards over (q, do) leaves dS+ of each chunk
//   segments where a row was cut into segments: the state before each of them
//   out, grad one CTA a chunk and head, 16 tokens a warp: scores by blocks of 16 x 16,
//            which pass from the accumulators of one product into the operands of
//            the next in registers
// The chunks do not wait for one another, so everything but the states' walk
// is as parallel as there are chunks.

#pragma once

#include <type_traits>

#include "cssd_internal.h"
#include "linattn_common.cuh"

namespace cssd {
namespace linattn {
namespace {

struct Shape {
    int T, H, G, N, P, nc;   // G: value heads per key head; nc: chunks of T tokens
    int seg, nseg;           // chunks a segment; segments
    int64_t g_row, g_tok;    // elements between batch rows and tokens of g (0: one decay a head)
    int BH;
    float scale;
};

// What a launch leaves for the others, in the workspace.
struct Scratch {
    float* states;   // [dir][b h][chunk][N][P]: before (dir 0) or after (dir 1) each chunk, without what came before its segment
    float* segs;     // [dir][b h][segment][N][P]: a segment's own state at its end, then the state before it
    float* seg_all;  // [dir][b h][segment]: its decay
    float* dec;      // [dir][b h][chunk]: decay from the segment's start to the chunk
};

// --------------------------------------------------------------- products
__host__ __device__ constexpr int imax(int a, int b) { return a > b ? a : b; }

// The sum over one chunk for 16 rows a warp,
//     acc = row_state (A S) + sum over blocks (A B^T, decayed) Z
// A, B and Z are tiles [token][column] of NPL planes, S a matrix [n][p] of SP planes that is filled by
// `fill` 64 rows at a time.  LOWER: the rows are the later tokens (o, dq), else the earlier ones (dk, dv).
// STRANS: A's columns are n and the outputs p (o, dv), else A's columns are p and the outputs n.
template <int NPL, int SP, int QP, int PP, int C, int KW, int OW, bool LOWER, bool STRANS>
struct Product {
    static constexpr int SN = STRANS ? KW : OW, SPW = STRANS ? OW : KW;  // S's widths: n, p
    static constexpr int RB = C / 16;

    template <typename Fill>
    static __device__ __forceinline__ void state(float (&acc)[OW / 8][4], uint32_t a, uint32_t s, int block, int kw, int ow,
                                                 int lane, Fill fill) {
        const int n = STRANS ? kw : ow;  // the state's rows
#pragma unroll
        for (int sl = 0; sl < SN / 64; ++sl) {
            if (64 * sl >= n) break;
            __syncthreads();
            fill(sl);
            __syncthreads();
            if constexpr (STRANS) {
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) {
                    const int k = 64 * sl + 16 * kt;
                    if (k >= kw) break;
                    uint32_t af[NPL][4];
#pragma unroll
                    for (int i = 0; i < NPL; ++i)
                        ldsm(af[i], lane_at<false>(a + i * C * pitch(KW), pitch(KW), 16 * block, k, lane));
#pragma unroll
                    for (int nt = 0; nt < OW / 16; ++nt) {
                        if (16 * nt >= ow) break;
#pragma unroll
                        for (int j = SP - 1; j >= 0; --j) {
                            uint32_t bf[4];
                            ldsm_t(bf, lane_at<false>(s + j * 64 * pitch(SPW), pitch(SPW), 16 * kt, 16 * nt, lane));
#pragma unroll
                            for (int i = NPL - 1; i >= 0; --i)
                                if (i + j < SP) {
                                    mma(acc[2 * nt], af[i], bf[0], bf[1]);
                                    mma(acc[2 * nt + 1], af[i], bf[2], bf[3]);
                                }
                        }
                    }
                }
            } else {
#pragma unroll
                for (int kt = 0; kt < KW / 16; ++kt) {
                    if (16 * kt >= kw) break;
                    uint32_t af[NPL][4];
#pragma unroll
                    for (int i = 0; i < NPL; ++i)
                        ldsm(af[i], lane_at<false>(a + i * C * pitch(KW), pitch(KW), 16 * block, 16 * kt, lane));
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) {
                        if (64 * sl + 16 * nt >= ow) break;
#pragma unroll
                        for (int j = SP - 1; j >= 0; --j) {
                            uint32_t bf[4];
                            ldsm(bf, lane_at<true>(s + j * 64 * pitch(SPW), pitch(SPW), 16 * nt, 16 * kt, lane));
#pragma unroll
                            for (int i = NPL - 1; i >= 0; --i)
                                if (i + j < SP) {
                                    mma(acc[8 * sl + 2 * nt], af[i], bf[0], bf[1]);
                                    mma(acc[8 * sl + 2 * nt + 1], af[i], bf[2], bf[3]);
                                }
                        }
                    }
                }
            }
        }
    }

    // `factor`: of every score.  `last`: blocks of tokens that there are.
    static __device__ __forceinline__ void pairs(float (&acc)[OW / 8][4], uint32_t a, uint32_t b, uint32_t z, int block, int kw,
                                                 int ow, int last, float factor, const Decays<C>& d, int lane) {
        const int r0 = 16 * block + lane / 4, c0 = 2 * (lane % 4);
        uint32_t keep[NPL == 1 ? KW / 16 : 1][4];
        if constexpr (NPL == 1)
#pragma unroll
            for (int kt = 0; kt < KW / 16; ++kt)
                if (16 * kt < kw) ldsm(keep[kt], lane_at<false>(a, pitch(KW), 16 * block, 16 * kt, lane));
        float row[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) row[e] = factor * (LOWER ? d.e[r0 + 8 * e] : d.f[r0 + 8 * e]);
#pragma unroll 1
        for (int o = LOWER ? 0 : block; o < (LOWER ? block + 1 : last); ++o) {
            float sc[2][4] = {};
#pragma unroll
            for (int kt = 0; kt < KW / 16; ++kt) {
                if (16 * kt >= kw) break;
                if constexpr (NPL == 1) {
                    uint32_t bf[4];
                    ldsm(bf, lane_at<true>(b, pitch(KW), 16 * o, 16 * kt, lane));
                    mma(sc[0], keep[kt], bf[0], bf[1]);
                    mma(sc[1], keep[kt], bf[2], bf[3]);
                } else {
                    uint32_t af[NPL][4];
#pragma unroll
                    for (int i = 0; i < NPL; ++i)
                        ldsm(af[i], lane_at<false>(a + i * C * pitch(KW), pitch(KW), 16 * block, 16 * kt, lane));
#pragma unroll
                    for (int j = NPL - 1; j >= 0; --j) {
                        uint32_t bf[4];
                        ldsm(bf, lane_at<true>(b + j * C * pitch(KW), pitch(KW), 16 * o, 16 * kt, lane));
#pragma unroll
                        for (int i = NPL - 1; i >= 0; --i)
                            if (i + j < QP) {
                                mma(sc[0], af[i], bf[0], bf[1]);
                                mma(sc[1], af[i], bf[2], bf[3]);
                            }
                    }
                }
            }
            // rows r0, r0 + 8; columns 16 o + c0, + 1, + 8, + 9
            if (o != block) {
                const float x = LOWER ? d.x[o][block] : d.x[block][o];
                const float x0 = row[0] * x, x1 = row[1] * x;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 c = *reinterpret_cast<const float2*>((LOWER ? d.f : d.e) + 16 * o + 8 * h + c0);
                    sc[h][0] *= x0 * c.x, sc[h][1] *= x0 * c.y;
                    sc[h][2] *= x1 * c.x, sc[h][3] *= x1 * c.y;
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = r0 + 8 * (e / 2), c = 16 * o + 8 * h + c0 + e % 2;
                        const int i = LOWER ? r : c, j = LOWER ? c : r;
                        const float m = factor * __expf((d.hi[i] - d.hi[j]) + (d.lo[i] - d.lo[j]));
                        sc[h][e] = i >= j ? sc[h][e] * m : 0.f;
                    }
            }
            uint32_t p[PP][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t w[PP];
                split<PP>(sc[u / 2][2 * (u % 2)], sc[u / 2][2 * (u % 2) + 1], w);
#pragma unroll
                for (int i = 0; i < PP; ++i) p[i][u] = w[i];
            }
#pragma unroll
            for (int nt = 0; nt < OW / 16; ++nt) {
                if (16 * nt >= ow) break;
#pragma unroll
                for (int j = NPL - 1; j >= 0; --j) {
                    uint32_t bf[4];
                    ldsm_t(bf, lane_at<false>(z + j * C * pitch(OW), pitch(OW), 16 * o, 16 * nt, lane));
#pragma unroll
                    for (int i = PP - 1; i >= 0; --i)
                        if (i + j < PP) {
                            mma(acc[2 * nt], p[i], bf[0], bf[1]);
                            mma(acc[2 * nt + 1], p[i], bf[2], bf[3]);
                        }
                }
            }
        }
    }
};

// The state before chunk c (dir 0) or after it (dir 1), as the states' walk left it.
struct StateAt {
    const float* own;   // null: none (the segment's first chunk)
    const float* seg;   // null: none
    float dec;
    __device__ __forceinline__ bool any() const { return own || seg; }
    __device__ __forceinline__ float4 at(int64_t i) const {
        float4 v = own ? __ldcs(reinterpret_cast<const float4*>(own + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (seg) {
            const float4 s = *reinterpret_cast<const float4*>(seg + i);
            v.x = fmaf(dec, s.x, v.x), v.y = fmaf(dec, s.y, v.y), v.z = fmaf(dec, s.z, v.z), v.w = fmaf(dec, s.w, v.w);
        }
        return v;
    }
};
__device__ __forceinline__ StateAt state_at(const Scratch& w, const Shape& sh, int dir, int64_t bh, int c, int live, bool start) {
    const int64_t np = (int64_t)sh.N * sh.P, row = (int64_t)dir * sh.BH + bh;
    const int walk = dir ? live - 1 - c : c, s = walk / sh.seg;
    StateAt r{w.states + (row * sh.nc + c) * np, nullptr, 0.f};
    if (sh.nseg == 1) {
        if (walk == 0 && !start) r.own = nullptr;
        return r;
    }
    if (walk % sh.seg == 0) r.own = nullptr;
    if (s > 0 || start) {
        r.seg = w.segs + (row * sh.nseg + s) * np;
        r.dec = w.dec[row * sh.nc + c];
    }
    return r;
}

// 64 rows of a state from row 64 sl on, as SP planes.
template <int SP, int PD>
__device__ __forceinline__ void fill_state(unsigned char* dst, const StateAt& st, int sl, const Shape& sh, int tid, int threads) {
    const int per = sh.P / 4, rows = min(64, sh.N - 64 * sl);
    for (int i = tid; i < rows * per; i += threads) {
        const int r = i / per, c = i - r * per;
        const float4 v = st.at((int64_t)(64 * sl + r) * sh.P + 4 * c);
        uint32_t x[SP], y[SP];
        split<SP>(v.x, v.y, x);
        split<SP>(v.z, v.w, y);
#pragma unroll
        for (int z = 0; z < SP; ++z)
            *reinterpret_cast<uint2*>(dst + z * 64 * pitch(PD) + r * pitch(PD) + 8 * c) = make_uint2(x[z], y[z]);
    }
}

// --------------------------------------------------------------- states
// A CTA has 64 columns p of a state (its columns never mix), a warp 16 rows n of
// them in registers, and takes every token's decayed key (three planes) times
// its value.  One more warp makes the next chunk's decays.
template <typename E, int ND, int C>
struct StatesSmem {
    static constexpr int NP = Type<E>::NP;
    static constexpr int X = NP * C * pitch(ND), Y = NP * C * pitch(64);
    static constexpr int STAGES = NP == 1 ? 2 : 1;  // (bfloat16 comes a chunk ahead)
    static constexpr int BYTES = STAGES * (X + Y);
    static constexpr int WARPS = ND / 16;
};

template <typename E, int ND, int C>
__global__ void __launch_bounds__(32 * (StatesSmem<E, ND, C>::WARPS + 1))
    states_kernel(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v, const E* __restrict__ dout,
                  const float* __restrict__ g, const int* __restrict__ lens, const float* h0, const float* dh_final,
                  float* h_final, float* gh0, Scratch w, Shape sh) {
    using M = StatesSmem<E, ND, C>;
    constexpr int NP = M::NP, NT = 32 * (M::WARPS + 1);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) Decays<C> tab[2];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int slices = (sh.P + 63) / 64, bh = blockIdx.x / slices, s = blockIdx.y, dir = blockIdx.z;
    const int p0 = 64 * (blockIdx.x % slices), cols = min(64, sh.P - p0);
    const int b = bh / sh.H, h = bh % sh.H, KH = sh.H / sh.G;
    const int len = row_len(lens, b, sh.T), live = (len + C - 1) / C;
    const int w0 = s * sh.seg, w1 = min(w0 + sh.seg, live);
    const int64_t np = (int64_t)sh.N * sh.P, row = (int64_t)dir * sh.BH + bh;
    const bool chain = warp < M::WARPS;
    const int n0 = 16 * warp;
    const bool mine = chain && n0 < sh.N, first = tid == 0 && p0 == 0;
    const E* xs = (dir ? q : k) + (int64_t)(h / sh.G) * sh.N;
    const E* ys = (dir ? dout : v) + (int64_t)h * sh.P + p0;
    const int64_t xst = (int64_t)KH * sh.N, yst = (int64_t)sh.H * sh.P;
    const float* gs = g + b * sh.g_row + h;
    auto chunk_of = [&](int i) { return dir ? live - 1 - i : i; };
    auto fetch = [&](int i) {
        const int c = chunk_of(i), n = min(len - c * C, C);
        const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C;
        unsigned char* at = smem + (M::STAGES == 2 ? (i & 1) * (M::X + M::Y) : 0);
        load_tile<E, ND>(at, C * pitch(ND), xs + t0 * xst, xst, C, n, sh.N, tid, NT);
        load_tile<E, 64>(at + M::X, C * pitch(64), ys + t0 * yst, yst, C, n, cols, tid, NT);
    };
    auto decays = [&](int i) {
        const int c = chunk_of(i);
        chunk_decays<C, false>(tab[i & 1], gs + (int64_t)c * C * sh.g_tok, sh.g_tok, min(len - c * C, C), lane);
    };
    float st[8][4];
    const float* start = dir ? dh_final : h0;
    auto each = [&](auto f) {  // pairs of the warp's part of the state
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int p = 8 * nt + 2 * (lane % 4);
                if (p < cols) f((int64_t)(n0 + lane / 4 + 4 * e) * sh.P + p0 + p, st[nt][e], st[nt][e + 1]);
            }
    };
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) st[nt][e] = 0.f;
    if (mine && sh.nseg == 1 && start)
        each([&](int64_t i, float& x, float& y) {
            const float2 a = *reinterpret_cast<const float2*>(start + bh * np + i);
            x = a.x, y = a.y;
        });
    if (w0 < w1) {
        if constexpr (M::STAGES == 2) {
            fetch(w0);
            cp_commit();
        }
        if (!chain) decays(w0);
    }
    float all = 1.f;  // decay since the segment's start
    for (int i = w0; i < w1; ++i) {
        if constexpr (M::STAGES == 2) {
            if (i + 1 < w1) fetch(i + 1);
            cp_commit();
            cp_wait<1>();
        } else {
            fetch(i);
        }
        __syncthreads();
        const Decays<C>& d = tab[i & 1];
        const int c = chunk_of(i);
        const bool empty = sh.nseg == 1 ? i == 0 && !start : i == w0;  // (not read by anyone)
        if (mine && !empty) {
            float* to = w.states + (row * sh.nc + c) * np;
            each([&](int64_t at, float x, float y) { *reinterpret_cast<float2*>(to + at) = make_float2(x, y); });
        }
        if (sh.nseg > 1 && first) w.dec[row * sh.nc + c] = all;
        if (!chain && i + 1 < w1) decays(i + 1);
        if (mine) {
            const uint32_t x = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + (M::STAGES == 2 ? (i & 1) * (M::X + M::Y) : 0);
            const uint32_t y = x + M::X;
            // the leading plane's products apart from the others': small terms are
            // not lost under large ones inside the matrix instruction
            float big[8][4] = {}, rest[8][4] = {};
            const float* wt = dir ? d.in : d.out;
            const float f = dir ? sh.scale : 1.f;
#pragma unroll 2
            for (int kt = 0; kt < C / 16; ++kt) {
                uint32_t raw[NP][4], a[3][4];
#pragma unroll
                for (int z = 0; z < NP; ++z) ldsm_t(raw[z], lane_at<true>(x + z * C * pitch(ND), pitch(ND), 16 * kt, n0, lane));
                const float2 u0 = *reinterpret_cast<const float2*>(wt + 16 * kt + 2 * (lane % 4));
                const float2 u1 = *reinterpret_cast<const float2*>(wt + 16 * kt + 8 + 2 * (lane % 4));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float e0 = 0.f, e1 = 0.f;
#pragma unroll
                    for (int z = NP - 1; z >= 0; --z) e0 += lo_f(raw[z][r]), e1 += hi_f(raw[z][r]);
                    uint32_t pl[3];
                    split<3>(e0 * (f * (r < 2 ? u0.x : u1.x)), e1 * (f * (r < 2 ? u0.y : u1.y)), pl);
                    a[0][r] = pl[0], a[1][r] = pl[1], a[2][r] = pl[2];
                }
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    if (16 * nt >= cols) break;
#pragma unroll
                    for (int j = NP - 1; j >= 0; --j) {
                        uint32_t bf[4];
                        ldsm_t(bf, lane_at<false>(y + j * C * pitch(64), pitch(64), 16 * kt, 16 * nt, lane));
#pragma unroll
                        for (int z = 2; z >= 0; --z)
                            if (z + j < 3) {
                                if (z + j == 0) {
                                    mma(big[2 * nt], a[z], bf[0], bf[1]);
                                    mma(big[2 * nt + 1], a[z], bf[2], bf[3]);
                                } else {
                                    mma(rest[2 * nt], a[z], bf[0], bf[1]);
                                    mma(rest[2 * nt + 1], a[z], bf[2], bf[3]);
                                }
                            }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) st[nt][e] = fmaf(d.all, st[nt][e], big[nt][e] + rest[nt][e]);
        }
        all *= d.all;
        __syncthreads();
    }
    float* to = sh.nseg > 1 ? w.segs + (row * sh.nseg + s) * np : (dir ? gh0 : h_final);
    if (sh.nseg == 1 && to) to += bh * np;
    if (mine && to && (sh.nseg == 1 || w0 < w1))
        each([&](int64_t at, float x, float y) { *reinterpret_cast<float2*>(to + at) = make_float2(x, y); });
    if (sh.nseg > 1 && first) w.seg_all[row * sh.nseg + s] = all;
}

// In place of each segment's own state, the state before it; the last goes out.
template <int C>
__global__ void __launch_bounds__(128) segments_kernel(const int* __restrict__ lens, const float* h0, const float* dh_final,
                                                       float* h_final, float* gh0, Scratch w, Shape sh) {
    const int64_t np = (int64_t)sh.N * sh.P;
    const int bh = blockIdx.y, dir = blockIdx.z;
    const int64_t row = (int64_t)dir * sh.BH + bh, i = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 4;
    if (i >= np) return;
    const int live = (row_len(lens, bh / sh.H, sh.T) + C - 1) / C, n = (live + sh.seg - 1) / sh.seg;
    const float* start = dir ? dh_final : h0;
    float4 r = start ? *reinterpret_cast<const float4*>(start + bh * np + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4* at = reinterpret_cast<float4*>(w.segs + row * sh.nseg * np + i);
    const float* all = w.seg_all + row * sh.nseg;
#pragma unroll 4
    for (int s = 0; s < n; ++s, at += np / 4) {
        const float4 own = *at;
        *at = r;
        const float d = all[s];
        r.x = fmaf(d, r.x, own.x), r.y = fmaf(d, r.y, own.y), r.z = fmaf(d, r.z, own.z), r.w = fmaf(d, r.w, own.w);
    }
    float* last = dir ? gh0 : h_final;
    if (last) *reinterpret_cast<float4*>(last + bh * np + i) = r;
}

// --------------------------------------------------------------- outputs
// A warp's 16 rows of `acc`, times `factor`, to tokens row0.. of a tensor with `stride` elements between
// tokens: n rows have values, those from n to `rows` are zeros.  16-bit types go
// through `stage` (16 rows of the warp's own) for whole 16-byte stores.
template <typename E, int OW>
__device__ __forceinline__ void put_rows(E* out, int64_t stride, const float (&acc)[OW / 8][4], float factor, unsigned char* stage,
                                         int ow, int n, int rows, int lane) {
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int nt = 0; nt < OW / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                alignas(4) E w[2] = {from_f<E>(factor * acc[nt][2 * e]), from_f<E>(factor * acc[nt][2 * e + 1])};
                *reinterpret_cast<uint32_t*>(stage + (lane / 4 + 8 * e) * pitch(OW) + 16 * nt + 4 * (lane % 4)) =
                    *reinterpret_cast<uint32_t*>(w);
            }
        __syncwarp();
        const int per = ow / 8;
        for (int i = lane; i < 16 * per; i += 32) {
            const int r = i / per, c = i - r * per;
            if (r < rows)
                __stcs(reinterpret_cast<uint4*>(out + r * stride + 8 * c),
                       r < n ? *reinterpret_cast<const uint4*>(stage + r * pitch(OW) + 16 * c) : make_uint4(0, 0, 0, 0));
        }
        __syncwarp();
    } else {
#pragma unroll
        for (int nt = 0; nt < OW / 8; ++nt) {
            if (8 * nt >= ow) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = lane / 4 + 8 * e;
                if (r < rows)
                    *reinterpret_cast<float2*>(out + r * stride + 8 * nt + 2 * (lane % 4)) =
                        r < n ? make_float2(factor * acc[nt][2 * e], factor * acc[nt][2 * e + 1]) : make_float2(0.f, 0.f);
            }
        }
    }
}

// The rows of a warp: blocks from both ends meet in one scheduler (warps w, w + 4), so that the
// triangle's work is even over the four.
template <int RB>
__device__ __forceinline__ int block_of(int warp) {
    return RB == 8 ? (warp < 4 ? warp : 11 - warp) : warp;
}

template <typename E, int ND, int PD, int C>
struct OutSmem {
    static constexpr int NP = Type<E>::NP, SP = NP == 3 ? 3 : 2;
    static constexpr int Q = 0, K = Q + NP * C * pitch(ND), V = K + NP * C * pitch(ND), S = V + NP * C * pitch(PD);
    static constexpr int BYTES = S + imax(SP * 64 * pitch(PD), sizeof(E) == 2 ? C * pitch(PD) : 0);
};

template <typename E, int ND, int PD, int C>
__global__ void __launch_bounds__(2 * C) out_kernel(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v,
                                                    const float* __restrict__ g, const int* __restrict__ lens, bool start,
                                                    E* __restrict__ o, Scratch w, Shape sh) {
    using M = OutSmem<E, ND, PD, C>;
    constexpr int NT = 2 * C;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) Decays<C> d;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int h = blockIdx.x % sh.H, bc = blockIdx.x / sh.H, c = bc % sh.nc, b = bc / sh.nc, KH = sh.H / sh.G;
    const int len = row_len(lens, b, sh.T), live = (len + C - 1) / C, n = min(len - c * C, C), rows = min(sh.T - c * C, C);
    const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C, bh = (int64_t)b * sh.H + h, os = (int64_t)sh.H * sh.P;
    E* orow = o + t0 * os + (int64_t)h * sh.P;
    if (n <= 0) {
        const int per = sh.P * (int)sizeof(E) / 16;
        for (int i = tid; i < rows * per; i += NT)
            reinterpret_cast<uint4*>(orow + (i / per) * os)[i % per] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int64_t ks = (int64_t)KH * sh.N, ko = t0 * ks + (int64_t)(h / sh.G) * sh.N;
    load_tile<E, ND>(smem + M::Q, C * pitch(ND), q + ko, ks, C, n, sh.N, tid, NT);
    load_tile<E, ND>(smem + M::K, C * pitch(ND), k + ko, ks, C, n, sh.N, tid, NT);
    load_tile<E, PD>(smem + M::V, C * pitch(PD), v + t0 * os + (int64_t)h * sh.P, os, C, n, sh.P, tid, NT);
    cp_commit();
    if (warp == 0) chunk_decays<C, true>(d, g + b * sh.g_row + h + (int64_t)c * C * sh.g_tok, sh.g_tok, n, lane);
    const StateAt st = state_at(w, sh, 0, bh, c, live, start);
    cp_wait<0>();
    __syncthreads();
    using Pr = Product<M::NP, M::SP, M::NP == 3 ? 3 : M::NP, M::SP, C, ND, PD, true, true>;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const int block = block_of<C / 16>(warp), r0 = 16 * block + lane / 4;
    float acc[PD / 8][4] = {};
    if (st.any()) {
        Pr::state(acc, base + M::Q, base + M::S, block, sh.N, sh.P, lane,
                  [&](int sl) { fill_state<M::SP, PD>(smem + M::S, st, sl, sh, tid, NT); });
        const float f0 = d.in[r0], f1 = d.in[r0 + 8];
#pragma unroll
        for (int nt = 0; nt < PD / 8; ++nt) acc[nt][0] *= f0, acc[nt][1] *= f0, acc[nt][2] *= f1, acc[nt][3] *= f1;
    }
    if (16 * block < n)
        Pr::pairs(acc, base + M::Q, base + M::K, base + M::V, block, sh.N, sh.P, 0, 1.f, d, lane);
    if (sizeof(E) == 2) __syncthreads();  // (the state's planes are read: the stage lies over them)
    put_rows<E, PD>(orow + 16 * block * os, os, acc, sh.scale, smem + M::S + 16 * block * pitch(PD), sh.P, n - 16 * block,
                    rows - 16 * block, lane);
}

// --------------------------------------------------------------- gradients
// Scores and states are split in three planes for dq and dk, whose sums make dg
// (a float32 result), in two for dv, which is rounded to 16 bits.
template <typename E, int ND, int PD, int C>
struct GradSmem {
    static constexpr int NP = Type<E>::NP;
    static constexpr int X = NP * C * pitch(ND), Y = NP * C * pitch(PD);
    static constexpr int Q = 0, K = X, V = 2 * X, DO = 2 * X + Y, S = 2 * X + 2 * Y;
    static constexpr int BYTES = S + imax(3 * 64 * pitch(PD), sizeof(E) == 2 ? C * pitch(imax(ND, PD)) : 0);
};

// Sum over a row's columns of the accumulators times a tile's values (rows r0 and r0 + 8), in every lane
// of the four that share the rows.
template <int NPL, int C, int W>
__device__ __forceinline__ float2 dot_rows(const float (&acc)[W / 8][4], const unsigned char* tile, int block, int width, int lane) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int nt = 0; nt < W / 8; ++nt) {
        if (8 * nt >= width) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int z = NPL - 1; z >= 0; --z) {
                const uint32_t v = *reinterpret_cast<const uint32_t*>(tile + z * C * pitch(W) + (16 * block + lane / 4 + 8 * e) * pitch(W) +
                                                                      16 * nt + 4 * (lane % 4));
                x += lo_f(v), y += hi_f(v);
            }
            float& s = e ? s1 : s0;
            s = fmaf(acc[nt][2 * e], x, s);
            s = fmaf(acc[nt][2 * e + 1], y, s);
        }
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        s1 += __shfl_xor_sync(0xffffffffu, s1, o);
    }
    return make_float2(s0, s1);
}

template <typename E, int ND, int PD, int C>
__global__ void __launch_bounds__(2 * C) grad_kernel(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v,
                                                     const E* __restrict__ dout, const float* __restrict__ g,
                                                     const int* __restrict__ lens, bool start, bool end, E* __restrict__ gq,
                                                     E* __restrict__ gk, E* __restrict__ gv, float* __restrict__ parts,
                                                     float* __restrict__ gg, float* __restrict__ gg_part, Scratch w, Shape sh) {
    using M = GradSmem<E, ND, PD, C>;
    constexpr int NT = 2 * C, NP = M::NP;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(16) Decays<C> d;
    __shared__ float s_r[C], s_state[C], s_dot[NT / 32];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int h = blockIdx.x % sh.H, bc = blockIdx.x / sh.H, c = bc % sh.nc, b = bc / sh.nc, KH = sh.H / sh.G;
    const int len = row_len(lens, b, sh.T), live = (len + C - 1) / C, n = min(len - c * C, C), rows = min(sh.T - c * C, C);
    const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C, bh = (int64_t)b * sh.H + h;
    const int64_t ks = (int64_t)KH * sh.N, ko = t0 * ks + (int64_t)(h / sh.G) * sh.N;
    const int64_t os = (int64_t)sh.H * sh.P, oo = t0 * os + (int64_t)h * sh.P;
    // with shared key heads a value head leaves its part in fp32
    const int64_t ps = (int64_t)sh.H * sh.N, po = t0 * ps + (int64_t)h * sh.N, pk = (int64_t)(gridDim.x / (sh.nc * sh.H)) * sh.T * ps;
    float* ggp = gg ? gg + t0 * sh.H + h : nullptr;
    if (n <= 0) {
        auto clear = [&](auto* at, int64_t stride, int width) {
            const int per = width * (int)sizeof(*at) / 16;
            for (int i = tid; i < rows * per; i += NT)
                reinterpret_cast<uint4*>(at + (i / per) * stride)[i % per] = make_uint4(0, 0, 0, 0);
        };
        clear(gv + oo, os, sh.P);
        if (parts) {
            clear(parts + po, ps, sh.N);
            clear(parts + pk + po, ps, sh.N);
        } else {
            clear(gq + ko, ks, sh.N);
            clear(gk + ko, ks, sh.N);
        }
        if (ggp)
            for (int i = tid; i < rows; i += NT) ggp[(int64_t)i * sh.H] = 0.f;
        if (gg_part && tid == 0) gg_part[blockIdx.x] = 0.f;
        return;
    }
    load_tile<E, ND>(smem + M::Q, C * pitch(ND), q + ko, ks, C, n, sh.N, tid, NT);
    load_tile<E, ND>(smem + M::K, C * pitch(ND), k + ko, ks, C, n, sh.N, tid, NT);
    load_tile<E, PD>(smem + M::V, C * pitch(PD), v + oo, os, C, n, sh.P, tid, NT);
    load_tile<E, PD>(smem + M::DO, C * pitch(PD), dout + oo, os, C, n, sh.P, tid, NT);
    cp_commit();
    if (warp == 0) chunk_decays<C, true>(d, g + b * sh.g_row + h + (int64_t)c * C * sh.g_tok, sh.g_tok, n, lane);
    const StateAt sb = state_at(w, sh, 0, bh, c, live, start), sa = state_at(w, sh, 1, bh, c, live, end);
    cp_wait<0>();
    __syncthreads();
    constexpr int QP = NP == 1 ? 1 : 3, VP = NP == 3 ? 3 : 2;
    using Pq = Product<NP, 3, QP, 3, C, PD, ND, true, false>;
    using Pk = Product<NP, 3, QP, 3, C, PD, ND, false, false>;
    using Pv = Product<NP, VP, QP, VP, C, ND, PD, false, true>;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const int block = block_of<C / 16>(warp), r0 = 16 * block + lane / 4, last = (n + 15) / 16;
    const bool on = block < last;
    const float scale = sh.scale;
    auto rows_times = [&](auto& acc, float f0, float f1) {
#pragma unroll
        for (auto& t : acc) t[0] *= f0, t[1] *= f0, t[2] *= f1, t[3] *= f1;
    };
    float2 rq;
    {
        float acc[ND / 8][4] = {};
        if (sb.any()) {
            Pq::state(acc, base + M::DO, base + M::S, block, sh.P, sh.N, lane,
                      [&](int sl) { fill_state<3, PD>(smem + M::S, sb, sl, sh, tid, NT); });
            rows_times(acc, scale * d.in[r0], scale * d.in[r0 + 8]);
        }
        if (on) Pq::pairs(acc, base + M::DO, base + M::V, base + M::K, block, sh.P, sh.N, 0, scale, d, lane);
        rq = dot_rows<NP, C, ND>(acc, smem + M::Q, block, sh.N, lane);
        __syncthreads();
        if (parts)
            put_rows<float, ND>(parts + po + 16 * block * ps, ps, acc, 1.f, nullptr, sh.N, n - 16 * block, rows - 16 * block, lane);
        else
            put_rows<E, ND>(gq + ko + 16 * block * ks, ks, acc, 1.f, smem + M::S + 16 * block * pitch(ND), sh.N, n - 16 * block,
                            rows - 16 * block, lane);
    }
    float dot = 0.f;  // <S, dS+>
    {
        float acc[ND / 8][4] = {};
        float2 own = make_float2(0.f, 0.f);
        if (sa.any()) {
            const bool both = sb.any();
            Pk::state(acc, base + M::V, base + M::S, block, sh.P, sh.N, lane, [&](int sl) {
                fill_state<3, PD>(smem + M::S, sa, sl, sh, tid, NT);
                if (both) {
                    const int per = sh.P / 4, top = min(64, sh.N - 64 * sl) * per;
                    for (int i = tid; i < top; i += NT) {
                        const int64_t at = (int64_t)64 * sl * sh.P + 4 * i;
                        const float4 x = sb.at(at), y = sa.at(at);
                        dot = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, dot))));
                    }
                }
            });
            rows_times(acc, d.out[r0], d.out[r0 + 8]);
            own = dot_rows<NP, C, ND>(acc, smem + M::K, block, sh.N, lane);
        }
        if (on) Pk::pairs(acc, base + M::V, base + M::DO, base + M::Q, block, sh.P, sh.N, last, scale, d, lane);
        const float2 rk = dot_rows<NP, C, ND>(acc, smem + M::K, block, sh.N, lane);
        if (lane % 4 == 0) {
            s_r[r0] = rq.x - rk.x, s_r[r0 + 8] = rq.y - rk.y;
            s_state[r0] = own.x, s_state[r0 + 8] = own.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) s_dot[warp] = dot;
        __syncthreads();
        if (parts)
            put_rows<float, ND>(parts + pk + po + 16 * block * ps, ps, acc, 1.f, nullptr, sh.N, n - 16 * block, rows - 16 * block, lane);
        else
            put_rows<E, ND>(gk + ko + 16 * block * ks, ks, acc, 1.f, smem + M::S + 16 * block * pitch(ND), sh.N, n - 16 * block,
                            rows - 16 * block, lane);
    }
    if (warp == 0 && (ggp || gg_part)) {
        float all = 0.f;
        for (int i = 0; i < NT / 32; ++i) all += s_dot[i];
        all *= d.all;
        // a lane's tokens, then the lanes after it
        constexpr int PER = C / 32;
        float r[PER], tail = 0.f, states = 0.f;
#pragma unroll
        for (int e = PER - 1; e >= 0; --e) {
            r[e] = s_r[PER * lane + e];
            tail += r[e];
            r[e] = tail;
            states += s_state[PER * lane + e];
        }
        float after = tail;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float t = __shfl_down_sync(0xffffffffu, after, o);
            if (lane + o < 32) after += t;
        }
        after -= tail;
#pragma unroll
        for (int o = 16; o; o >>= 1) states += __shfl_xor_sync(0xffffffffu, states, o);
        const float leaves = all + states;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = PER * lane + e;
            const float x = i < n ? leaves + (after + r[e]) : 0.f;
            sum += x;
            if (ggp && i < rows) ggp[(int64_t)i * sh.H] = x;
        }
        if (gg_part) {
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) gg_part[blockIdx.x] = sum;
        }
    }
    {
        float acc[PD / 8][4] = {};
        if (sa.any()) {
            Pv::state(acc, base + M::K, base + M::S, block, sh.N, sh.P, lane,
                      [&](int sl) { fill_state<VP, PD>(smem + M::S, sa, sl, sh, tid, NT); });
            rows_times(acc, d.out[r0], d.out[r0 + 8]);
        }
        if (on) Pv::pairs(acc, base + M::K, base + M::Q, base + M::DO, block, sh.N, sh.P, last, scale, d, lane);
        if (sizeof(E) == 2) __syncthreads();
        put_rows<E, PD>(gv + oo + 16 * block * os, os, acc, 1.f, smem + M::S + 16 * block * pitch(PD), sh.P, n - 16 * block,
                        rows - 16 * block, lane);
    }
}

// Shared key heads: the sum over a key head's value heads, in their order.
template <typename E>
__global__ void __launch_bounds__(256) join_kernel(const float* __restrict__ parts, E* __restrict__ gq, E* __restrict__ gk,
                                                   int64_t vectors, int64_t part, int G, int N) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // four columns of a token and key head
    if (i >= vectors) return;
    const int64_t row = i / (N / 4);
    const int c = (int)(i % (N / 4)) * 4;
    const float* at = parts + blockIdx.y * part + row * G * N + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u = 0; u < G; ++u) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(at + (int64_t)u * N));
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    E* to = (blockIdx.y ? gk : gq) + row * N + c;
    alignas(16) E e[4] = {from_f<E>(s.x), from_f<E>(s.y), from_f<E>(s.z), from_f<E>(s.w)};
    if constexpr (sizeof(E) == 2)
        *reinterpret_cast<uint2*>(to) = *reinterpret_cast<uint2*>(e);
    else
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<uint4*>(e);
}

// One decay a head: its gradient from the chunks' sums [chunk of every row][H], in 64 bits.
__global__ void __launch_bounds__(128) join_g_kernel(const float* __restrict__ part, float* __restrict__ gg, int64_t chunks, int H) {
    __shared__ double red[128];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < chunks; i += 128) s += (double)part[i * H + blockIdx.x];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int o = 64; o; o >>= 1) {
        if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) gg[blockIdx.x] = (float)red[0];
}

// --------------------------------------------------------------- launches
// The chunk: what leaves a chunk's tiles of the gradients and 64 rows of a state
// room in one SM's shared memory.
template <typename E, int ND, int PD>
constexpr int chunk_tokens() {
    return Type<E>::NP == 1 ? 128 : Type<E>::NP == 2 ? 64 : imax(ND, PD) == 64 ? 64 : 32;
}
int chunk_of(const LinattnArgs& a) {
    if (a.dtype == CSSD_BF16) return 128;
    if (a.dtype == CSSD_F16) return 64;
    return a.N <= 64 && a.P <= 64 ? 64 : 32;
}

constexpr int kStateCtas = 304;  // CTAs that the states' walk aims at: two an SM

Shape shape_of(const LinattnArgs& a, int dirs) {
    Shape sh{};
    const int C = chunk_of(a);
    sh.T = (int)a.T, sh.H = (int)a.H, sh.G = (int)(a.H / a.KH), sh.N = (int)a.N, sh.P = (int)a.P;
    sh.nc = (int)((a.T + C - 1) / C);
    sh.BH = (int)(a.Bz * a.H);
    const int64_t rows = a.Bz * a.H * dirs * ((a.P + 63) / 64);
    const int64_t want = rows >= kStateCtas ? 1 : (kStateCtas + rows - 1) / rows;
    sh.seg = (int)((sh.nc + want - 1) / want);
    sh.nseg = (sh.nc + sh.seg - 1) / sh.seg;
    sh.g_row = a.g_tokens ? a.T * a.H : 0;
    sh.g_tok = a.g_tokens ? a.H : 0;
    sh.scale = a.scale;
    return sh;
}

size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

size_t scratch_bytes(const LinattnArgs& a, int dirs) {
    const Shape sh = shape_of(a, dirs);
    const size_t rows = (size_t)dirs * sh.BH, np = (size_t)sh.N * sh.P * 4;
    size_t n = up(rows * sh.nc * np);
    if (sh.nseg > 1) n += up(rows * sh.nseg * np) + up(rows * sh.nseg * 4) + up(rows * sh.nc * 4);
    return n;
}
Scratch scratch_of(const LinattnArgs& a, int dirs, void* ws) {
    const Shape sh = shape_of(a, dirs);
    const size_t rows = (size_t)dirs * sh.BH, np = (size_t)sh.N * sh.P * 4;
    unsigned char* p = static_cast<unsigned char*>(ws);
    Scratch s{};
    auto take = [&](size_t n) {
        float* at = reinterpret_cast<float*>(p);
        p += up(n);
        return at;
    };
    s.states = take(rows * sh.nc * np);
    if (sh.nseg > 1) {
        s.segs = take(rows * sh.nseg * np);
        s.seg_all = take(rows * sh.nseg * 4);
        s.dec = take(rows * sh.nc * 4);
    }
    return s;
}

template <typename E, int ND, int PD>
cudaError_t run_states(const LinattnArgs& a, int dirs, const Scratch& w, const Shape& sh, cudaStream_t st) {
    constexpr int C = chunk_tokens<E, ND, PD>();
    using M = StatesSmem<E, ND, C>;
    auto* kernel = states_kernel<E, ND, C>;
    cudaError_t e = delta::allow<states_kernel<E, ND, C>>(M::BYTES);
    if (e != cudaSuccess) return e;
    kernel<<<dim3(sh.BH * ((sh.P + 63) / 64), sh.nseg, dirs), 32 * (M::WARPS + 1), M::BYTES, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.v), static_cast<const E*>(a.dout), a.g,
        a.lens, a.h0, a.dh_final, a.h_final, a.gh0, w, sh);
    if (sh.nseg > 1)
        segments_kernel<C><<<dim3((sh.N * sh.P + 511) / 512, sh.BH, dirs), 128, 0, st>>>(a.lens, a.h0, a.dh_final, a.h_final, a.gh0, w, sh);
    return cudaGetLastError();
}

template <typename E, int ND, int PD>
cudaError_t forward(const LinattnArgs& a, void* ws, cudaStream_t st) {
    constexpr int C = chunk_tokens<E, ND, PD>();
    using M = OutSmem<E, ND, PD, C>;
    const Shape sh = shape_of(a, 1);
    const Scratch w = scratch_of(a, 1, ws);
    cudaError_t e = run_states<E, ND, PD>(a, 1, w, sh, st);
    if (e == cudaSuccess) e = delta::allow<out_kernel<E, ND, PD, C>>(M::BYTES);
    if (e != cudaSuccess) return e;
    out_kernel<E, ND, PD, C><<<(unsigned)(sh.BH * sh.nc), 2 * C, M::BYTES, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.v), a.g, a.lens, a.h0 != nullptr,
        static_cast<E*>(a.o), w, sh);
    return cudaGetLastError();
}

size_t parts_bytes(const LinattnArgs& a) { return a.H == a.KH ? 0 : up((size_t)2 * a.Bz * a.T * a.H * a.N * 4); }

template <typename E, int ND, int PD>
cudaError_t backward(const LinattnArgs& a, void* ws, cudaStream_t st) {
    constexpr int C = chunk_tokens<E, ND, PD>();
    using M = GradSmem<E, ND, PD, C>;
    const Shape sh = shape_of(a, 2);
    const Scratch w = scratch_of(a, 2, ws);
    unsigned char* rest = static_cast<unsigned char*>(ws) + scratch_bytes(a, 2);
    float* parts = parts_bytes(a) ? reinterpret_cast<float*>(rest) : nullptr;
    float* gg_part = a.gg && !a.g_tokens ? reinterpret_cast<float*>(rest + parts_bytes(a)) : nullptr;
    cudaError_t e = run_states<E, ND, PD>(a, 2, w, sh, st);
    if (e == cudaSuccess) e = delta::allow<grad_kernel<E, ND, PD, C>>(M::BYTES);
    if (e != cudaSuccess) return e;
    grad_kernel<E, ND, PD, C><<<(unsigned)(sh.BH * sh.nc), 2 * C, M::BYTES, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.v), static_cast<const E*>(a.dout), a.g,
        a.lens, a.h0 != nullptr, a.dh_final != nullptr, static_cast<E*>(a.gq), static_cast<E*>(a.gk), static_cast<E*>(a.gv), parts,
        a.g_tokens ? a.gg : nullptr, gg_part, w, sh);
    if (parts) {
        const int64_t vectors = a.Bz * a.T * a.KH * (a.N / 4);
        join_kernel<E><<<dim3((unsigned)((vectors + 255) / 256), 2), 256, 0, st>>>(parts, static_cast<E*>(a.gq), static_cast<E*>(a.gk),
                                                                                  vectors, a.Bz * a.T * a.H * a.N, sh.G, sh.N);
    }
    if (gg_part) join_g_kernel<<<sh.H, 128, 0, st>>>(gg_part, a.gg, a.Bz * sh.nc, sh.H);
    return cudaGetLastError();
}

// Calls f with the widths' tiles (64 or 128 columns).
template <typename F>
cudaError_t by_widths(const LinattnArgs& a, F f) {
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (a.N <= 64) return a.P <= 64 ? f(I64(), I64()) : f(I64(), I128());
    return a.P <= 64 ? f(I128(), I64()) : f(I128(), I128());
}
template <typename E>
cudaError_t forward_of(const LinattnArgs& a, void* ws, cudaStream_t st) {
    return by_widths(a, [&](auto n, auto p) { return forward<E, decltype(n)::value, decltype(p)::value>(a, ws, st); });
}
template <typename E>
cudaError_t backward_of(const LinattnArgs& a, void* ws, cudaStream_t st) {
    return by_widths(a, [&](auto n, auto p) { return backward<E, decltype(n)::value, decltype(p)::value>(a, ws, st); });
}

}  // namespace
}  // namespace linattn
}  // namespace cssd
