// Linear attention with a decay for each head, over a sequence:
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// in chunks of C tokens.  With G_i the running sum of g in a chunk and
// M_ij = e^{G_i - G_j} (i >= j),
//     o_i   = scale (e^{G_i} q_i S + sum_j M_ij (q_i.k_j) v_j)
//     S+    = e^{G_end} S + sum_j e^{G_end - G_j} k_j v_j^T
// and, dS+ being the gradient of the state that leaves the chunk and
// W_ij = scale M_ij (q_i.k_j) (do_i.v_j),
//     dq_i  = scale (e^{G_i} do_i S^T + sum_j M_ij (do_i.v_j) k_j)
//     dk_j  = e^{G_end - G_j} v_j dS+^T + scale sum_i M_ij (do_i.v_j) q_i
//     dv_j  = e^{G_end - G_j} k_j dS+   + scale sum_i M_ij (q_i.k_j) do_i
//     dS    = e^{G_end} dS+ + sum_i scale e^{G_i} q_i do_i^T
//     dg_t  = e^{G_end} <S, dS+> + sum_{j < t} b_j + sum_{u >= t} (a_u + sum_j W_uj - sum_i W_iu)
// with a_u, b_j the first terms' shares of q_u.dq_u and k_j.dk_j, and W without its diagonal.  (dg_t = <e^{g_t}
// S_{t-1}, dL/dS_t>, every pair and every state's term that spans t.  The pairs after t cancel in the sum up to its
// rounding, about 2^-24 of their sizes; with the diagonal, which spans no decay, that would be 2^-24 of the tokens' own
// writes: a head with g = -10 was off by 0.2 to 0.7 % in the 2-norm.  W is made from the scores in fp32, so that dg
// does not see the splitting of the operands.)
//
// Two kernels:
//   states   walks the chunks of a row and head and leaves the state before each chunk; for the gradients the same
//            walk backwards over (q, do) leaves dS+ of each chunk.  A row is cut into up to 8 segments, a cluster of
//            CTAs, which tell one another the segments' own states at the end.
//   out, grad one CTA a chunk and head, 16 tokens a warp: scores by blocks of 16 x 16, which pass from the
//            accumulators of one product into the operands of the next in registers
// The chunks do not wait for one another, so everything but the states' walk is as parallel as there are chunks.
//
// What a value is rounded to: inputs are exact in their planes; decayed keys, and states for dq and dk, have three
// (24 bits: float32 results, the last state, dS and dg, come from them); scores, and states for 16-bit results,
// two (16 bits, 2^-18 of each term at most, far below the result's own rounding).  One plane of the scores
// would add an error as large as the output's own rounding and made the forward no faster (67.3 us against 67.3).
//
// Most products are warp-level matrix instructions, whose rate here is 581 TFLOP/s (measured), a third of the
// tcgen05 ones': with it the 64/64 forward of 4 x 2048 x 24 needs 22 us of tensor time beside 34 us of its
// memory traffic (the states among it), in exchange for scores that never leave the registers, three CTAs an SM
// and no barrier inside a chunk's products.  The state's products of the wide gradients are tcgen05 ones: there every
// warp would read all of a state from shared memory for its 16 rows.
//
// Measured, bf16 (a call among others of its kind): forward 4 x 2048 x 24, 64/64 66 us (walk 29, outputs 37: half of
// it the loads' latency at three CTAs an SM; without any products 41 us); 1 x 16384 x 32, 128/64 298 us (walk 119, 1 GB
// moved with the states); gradients 4 x 2048 x 24, 64/64 187 us (walk 48, grad_kernel 139, 96 bytes a thread of spilled
// registers); 4 x 1501 x 16 on 8 key heads, 128/128, rows of random lengths, 165 to 205 us (at 82 % of the tokens 198:
// walk 52, grad_kernel 130, sum over shared heads 23).
#pragma once

#include <type_traits>

#include "cssd_internal.h"
#include "linattn_common.cuh"
#include "tcgen05.cuh"

namespace cssd {
namespace linattn {
namespace {

struct Shape {
    int T, H, G, N, P, nc;   // G: value heads per key head; nc: chunks of T tokens
    int seg, nseg;           // chunks a segment; segments (at most kMostSegments)
    int64_t g_row, g_tok;    // elements between batch rows and tokens of g (0: one decay a head)
    int BH;
    float scale;
    Divisor by_h, by_nc, by_slices;
};
constexpr int kMostSegments = 8;  // CTAs of a cluster

// What the states' walk leaves for the others, in the workspace.
struct Scratch {
    float* states;   // [dir][b h][chunk][N][P]: before (dir 0) or after (dir 1) each chunk, without what came before its segment
    float* ends;     // [dir][b h][segment][N][P]: a segment's own state at its end
    float* starts;   // [dir][b h][segment][N][P]: the state before it
    float* seg_all;  // [dir][b h][segment]: its decay
    float* dec;      // [dir][b h][chunk]: decay from the segment's start to the chunk
    void* decays;    // [b h][chunk] Decays<C>
};

__host__ __device__ constexpr int imax(int a, int b) { return a > b ? a : b; }
__host__ __device__ constexpr int imin(int a, int b) { return a < b ? a : b; }

// --------------------------------------------------------------- products
constexpr int NT = 256;  // threads of out and grad

// A warp's part of a chunk: 16 rows and, with fewer than eight blocks of rows, a share of the columns.  The two
// warps of a scheduler (w, w + 4) get blocks from both ends, so that the triangle's work is even over the four.
template <int C>
struct Part {
    static constexpr int RB = C / 16, CS = 8 / RB;  // blocks of rows, shares of the columns
    int block, share;
    __device__ __forceinline__ explicit Part(int warp) {
        if (RB == 8)
            block = warp < 4 ? warp : 11 - warp, share = 0;
        else if (RB == 4)
            block = warp < 4 ? warp : 7 - warp, share = warp / 4;
        else
            block = (warp ^ warp / 4) & 1, share = warp / 2;
    }
};

// What float32 results of tensors in more than one plane come from (APART): the products other than the leading planes'
// are summed apart and added at the end.  The matrix instruction drops what lies below its sum's last bit, at every one
// of its steps (in one sum, float32 outputs of 128/128 were off by 1.1e-6 in the 2-norm where plain fp32 arithmetic is off
// by 2.5e-7, and dg of float16 tensors by 0.7 to 1.0e-6, now 2 to 3e-7; the latter's times are the same within 1 %).
template <bool APART, int N>
struct Rest {
    float v[APART ? N : 1][4];
    __device__ __forceinline__ Rest() {
#pragma unroll
        for (auto& t : v)
#pragma unroll
            for (float& x : t) x = 0.f;
    }
    // where the product of planes i and j of sum n goes
    __device__ __forceinline__ float (&of(float (&acc)[N][4], int n, int ij))[4] { return APART && ij > 0 ? v[APART ? n : 0] : acc[n]; }
    __device__ __forceinline__ void add_to(float (&acc)[N][4]) const {
        if constexpr (APART)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][e] += v[n][e];
    }
};

// acc += A S (or A S^T) of 16 rows and columns col0.. (CW of them): one slice of 64 of the state's rows n, as SP
// planes at `s`.  A is a tile [token][column] of NPL planes.
//   TRANS   A's columns are n, the outputs are p:  acc[., p] += sum_n A[., n] S[n][p]
//   else    A's columns are p, the outputs are n:  acc[., n] += sum_p A[., p] S[n][p], n of this slice
template <int NPL, int SP, int C, int KW, int OW, int CW, bool TRANS>
__device__ __forceinline__ void times_state(float (&acc)[CW / 8][4], uint32_t a, uint32_t s, int block, int col0, int sl, int kw,
                                            int ow, int lane) {
    using TA = Tile<false, C, KW>;
    using TS = Tile<false, 64, TRANS ? OW : KW>;
    constexpr int KT = TRANS ? imin(4, KW / 16) : KW / 16;
    const int k0 = TRANS ? 64 * sl : 0;
    Rest<(NPL > 1 && SP == 3), CW / 8> rest;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
        if (k0 + 16 * kt >= kw) break;
        uint32_t af[NPL][4];
#pragma unroll
        for (int i = 0; i < NPL; ++i) ldsm(af[i], TA::template at<false>(a + i * TA::PLANE, block, k0 + 16 * kt, lane));
        // (columns inside: a sum is added to again only after all the others)
#pragma unroll
        for (int j = SP - 1; j >= 0; --j) {
            uint32_t bf[CW / 16][4];
#pragma unroll
            for (int nt = 0; nt < CW / 16; ++nt) {
                const int col = col0 + 16 * nt;
                if (col >= ow) break;
                if (!TRANS && col / 64 != sl) continue;
                if (TRANS)
                    ldsm_t(bf[nt], TS::template at<false>(s + j * TS::PLANE, kt, col, lane));
                else
                    ldsm(bf[nt], TS::template at<true>(s + j * TS::PLANE, col % 64 / 16, 16 * kt, lane));
            }
#pragma unroll
            for (int i = NPL - 1; i >= 0; --i)
                if (i + j < SP)
#pragma unroll
                    for (int nt = 0; nt < CW / 16; ++nt) {
                        const int col = col0 + 16 * nt;
                        if (col >= ow) break;
                        if (!TRANS && col / 64 != sl) continue;
                        mma(rest.of(acc, 2 * nt, i + j), af[i], bf[nt][0], bf[nt][1]);
                        mma(rest.of(acc, 2 * nt + 1, i + j), af[i], bf[nt][2], bf[nt][3]);
                    }
        }
    }
    rest.add_to(acc);
}

// The operands A of the scores: kept in registers where they are one plane of at most 64 columns.
template <int NPL, int C, int KW, bool TC>
struct Rows {
    using TA = Tile<TC, C, KW>;
    static constexpr bool KEEP = NPL == 1 && KW <= 64;
    uint32_t f[KEEP ? KW / 16 : 1][4];
    uint32_t at;
    __device__ __forceinline__ Rows(uint32_t a, int block, int kw, int lane) : at(TA::template at<false>(a, block, 0, lane)) {
        if constexpr (KEEP)
#pragma unroll
            for (int kt = 0; kt < KW / 16; ++kt)
                if (16 * kt < kw) ldsm(f[kt], at + TA::STEP * kt);
    }
};
// sc = A B^T for the warp's 16 rows and the 16 tokens of block `o` of B.
template <int NPL, int QP, int C, int KW, bool TC>
__device__ __forceinline__ void scores(float (&sc)[2][4], const Rows<NPL, C, KW, TC>& a, uint32_t b, int o, int kw, int lane) {
    using TB = Tile<TC, C, KW>;
    const uint32_t at = TB::template at<true>(b, o, 0, lane);
    Rest<(NPL > 1 && QP == 3), 2> rest;
    if (NPL > 1)
#pragma unroll
        for (auto& t : sc) t[0] = t[1] = t[2] = t[3] = 0.f;
#pragma unroll
    for (int kt = 0; kt < KW / 16; ++kt) {
        if (16 * kt >= kw) break;
        if constexpr (NPL == 1) {
            uint32_t bf[4], af[4];
            ldsm(bf, at + TB::STEP * kt);
            if constexpr (Rows<NPL, C, KW, TC>::KEEP) {
#pragma unroll
                for (int e = 0; e < 4; ++e) af[e] = a.f[kt][e];
            } else {
                ldsm(af, a.at + TB::STEP * kt);
            }
            if (kt == 0) {
                mma_first(sc[0], af, bf[0], bf[1]);
                mma_first(sc[1], af, bf[2], bf[3]);
            } else {
                mma(sc[0], af, bf[0], bf[1]);
                mma(sc[1], af, bf[2], bf[3]);
            }
        } else {
            uint32_t af[NPL][4];
#pragma unroll
            for (int i = 0; i < NPL; ++i) ldsm(af[i], a.at + i * TB::PLANE + TB::STEP * kt);
#pragma unroll
            for (int j = NPL - 1; j >= 0; --j) {
                uint32_t bf[4];
                ldsm(bf, at + j * TB::PLANE + TB::STEP * kt);
#pragma unroll
                for (int i = NPL - 1; i >= 0; --i)
                    if (i + j < QP) {
                        mma(rest.of(sc, 0, i + j), af[i], bf[0], bf[1]);
                        mma(rest.of(sc, 1, i + j), af[i], bf[2], bf[3]);
                    }
            }
        }
    }
    rest.add_to(sc);
}
// The factors scale M of a block's pairs: the warp's rows (the later tokens if LOWER, else the earlier ones) with
// the tokens of block `o`; 0 where the pair is none.  `row`: scale times the rows' own factors.
template <int C, bool LOWER, bool DIAG>
__device__ __forceinline__ void pair_factors(float (&m)[2][4], const Decays<C>& d, int block, int o, const float (&row)[2], float scale,
                                             int lane) {
    const int c0 = 16 * o + 2 * (lane % 4);
    if constexpr (!DIAG) {
        const float x = LOWER ? d.x[o][block] : d.x[block][o];
        const float x0 = row[0] * x, x1 = row[1] * x;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 c = *reinterpret_cast<const float2*>((LOWER ? d.f : d.e) + c0 + 8 * h);
            m[h][0] = x0 * c.x, m[h][1] = x0 * c.y, m[h][2] = x1 * c.x, m[h][3] = x1 * c.y;
        }
    } else {
        const int r0 = 16 * block + lane / 4;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = r0 + 8 * (e / 2), c = c0 + 8 * h + e % 2, i = LOWER ? r : c, j = LOWER ? c : r;
                m[h][e] = i >= j ? scale * __expf((d.hi[i] - d.hi[j]) + (d.lo[i] - d.lo[j])) : 0.f;
            }
    }
}
template <int C, bool LOWER>
__device__ __forceinline__ void row_factors(float (&row)[2], const Decays<C>& d, int block, float scale, int lane) {
    const float* t = (LOWER ? d.e : d.f) + 16 * block + lane / 4;
    row[0] = scale * t[0], row[1] = scale * t[8];
}
__device__ __forceinline__ void multiply(float (&sc)[2][4], const float (&m)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[h][e] *= m[h][e];
}
// acc += P Z for columns col0.. of Z's 16 tokens of block `o`; the scores P, split in PP planes, are the operand as
// they lie.
template <int NPL, int PP, int C, int OW, int CW, bool TC>
__device__ __forceinline__ void times_tokens(float (&acc)[CW / 8][4], const float (&sc)[2][4], uint32_t z, int col0, int o, int ow, int lane) {
    uint32_t p[PP][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        uint32_t w[PP];
        split<PP>(sc[u / 2][2 * (u % 2)], sc[u / 2][2 * (u % 2) + 1], w);
#pragma unroll
        for (int i = 0; i < PP; ++i) p[i][u] = w[i];
    }
    using TZ = Tile<TC, C, OW>;
    const uint32_t at = TZ::template at<false>(z, o, col0, lane);
    constexpr int NG = imin(CW / 16, 4);  // 64 columns at a time
    Rest<NPL == 3, CW / 8> rest;
#pragma unroll
    for (int n0 = 0; n0 < CW / 16; n0 += NG)
#pragma unroll
        for (int j = NPL - 1; j >= 0; --j) {
            uint32_t bf[NG][4];
#pragma unroll
            for (int nt = 0; nt < NG; ++nt)
                if (col0 + 16 * (n0 + nt) < ow) ldsm_t(bf[nt], at + j * TZ::PLANE + TZ::STEP * (n0 + nt));
#pragma unroll
            for (int i = PP - 1; i >= 0; --i)
                if (i + j < PP)
#pragma unroll
                    for (int nt = 0; nt < NG; ++nt)
                        if (col0 + 16 * (n0 + nt) < ow) {
                            mma(rest.of(acc, 2 * (n0 + nt), i + j), p[i], bf[nt][0], bf[nt][1]);
                            mma(rest.of(acc, 2 * (n0 + nt) + 1, i + j), p[i], bf[nt][2], bf[nt][3]);
                        }
        }
    rest.add_to(acc);
}
// acc = sum over the blocks at or before the warp's of (A B^T, decayed) Z.
template <int NPL, int QP, int PP, int C, int KW, int OW, int CW, bool TC>
__device__ __forceinline__ void earlier_pairs(float (&acc)[CW / 8][4], uint32_t a, uint32_t b, uint32_t z, int block, int col0, int kw, int ow,
                                              float scale, const Decays<C>& d, int lane) {
    const Rows<NPL, C, KW, TC> rows(a, block, kw, lane);
    float row[2];
    row_factors<C, true>(row, d, block, scale, lane);
    auto with = [&](int o, auto diag) {
        constexpr bool DIAG = decltype(diag)::value;
        float sc[2][4], m[2][4];
        scores<NPL, QP, C, KW, TC>(sc, rows, b, o, kw, lane);
        pair_factors<C, true, DIAG>(m, d, block, o, row, scale, lane);
        if constexpr (DIAG) {  // (a score that is not wanted may be anything)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[h][e] = lane / 4 + 8 * (e / 2) >= 8 * h + 2 * (lane % 4) + e % 2 ? sc[h][e] : 0.f;
        }
        multiply(sc, m);
        times_tokens<NPL, PP, C, OW, CW, TC>(acc, sc, z, col0, o, ow, lane);
    };
#pragma unroll 1
    for (int o = 0; o < block; ++o) with(o, std::false_type());
    with(block, std::true_type());
}
template <int N>
__device__ __forceinline__ void scale_rows(float (&acc)[N][4], float f0, float f1) {
#pragma unroll
    for (auto& t : acc) t[0] *= f0, t[1] *= f0, t[2] *= f1, t[3] *= f1;
}

// The state before chunk c (dir 0) or after it (dir 1), as the states' walk left it.
struct StateAt {
    const float* own;   // null: none (the segment's first chunk)
    const float* seg;   // null: none
    float dec;
    __device__ __forceinline__ bool any() const { return own || seg; }
    __device__ __forceinline__ float4 at(int i) const {
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
    const int walk = dir ? live - 1 - c : c;
    StateAt r{w.states + (row * sh.nc + c) * np, nullptr, 0.f};
    if (sh.nseg == 1) {
        if (walk == 0 && !start) r.own = nullptr;
        return r;
    }
    const int s = walk / sh.seg;
    if (walk % sh.seg == 0) r.own = nullptr;
    if (s > 0 || start) {
        r.dec = w.dec[row * sh.nc + c];
        if (r.dec != 0.f) r.seg = w.starts + (row * sh.nseg + s) * np;  // (else nothing is left of it; NaN is not 0)
    }
    return r;
}

// 64 rows of a state from row 64 sl on: fetched into registers, and put as SP planes of a tile of 64 rows n.
template <int SP, int PD, bool TC>
struct StateTile {
    static constexpr int PER = PD / 4, STEP = NT / PER, K = 64 / STEP;
    float4 v[K];
    __device__ __forceinline__ void fetch(const StateAt& st, int sl, int N, int P, int tid) {
        const int r = 64 * sl + tid / PER, c = 4 * (tid % PER);
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] = c < P && r + STEP * k < N ? st.at((r + STEP * k) * P + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void put(unsigned char* dst, int tid) const {
        const int c = 4 * (tid % PER);
        constexpr int ROW = TC ? 16 : pitch(PD);
        unsigned char* at = dst + (TC ? c / 8 * group_bytes(64) + c % 8 * 2 : 2 * c) + tid / PER * ROW;
#pragma unroll
        for (int k = 0; k < K; ++k, at += ROW * STEP) {
            uint32_t x[SP], y[SP];
            split<SP>(v[k].x, v[k].y, x);
            split<SP>(v[k].z, v[k].w, y);
#pragma unroll
            for (int z = 0; z < SP; ++z) *reinterpret_cast<uint2*>(at + z * Tile<TC, 64, PD>::PLANE) = make_uint2(x[z], y[z]);
        }
    }
};

// --------------------------------------------------------------- the state's products on tcgen05
// Chunks of 128 tokens (bfloat16): [128 tokens] x [a state's 64 rows a time] into tensor memory, from the tiles as
// they lie, beside the warps' work on the scores.  A warp gets its 16 rows in the layout of its own sums.
constexpr long long kLinattnWait = 4000000000LL;  // ~2 s at 2 GHz

// One thread.  TRANS: D[., p] (+)= A[., n] S[n][p] over the slice's n; else D[., n of the slice] = A[., p] S[n][p].
template <int KW, int OW, int SP, bool TRANS>
__device__ __forceinline__ void issue_state(uint32_t tmem, uint32_t a, uint32_t s, int sl, int kw) {
    constexpr int PLANE = plane_bytes(64, TRANS ? OW : KW), KT = TRANS ? 4 : KW / 16, N = TRANS ? OW : 64;
    constexpr int GA = group_bytes(128), GS = group_bytes(64);
    // D fp32, A and B bfloat16, B's columns contiguous (TRANS) or its sum
    constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (TRANS ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
    const int k0 = TRANS ? 64 * sl : 0;
    if (!TRANS) tmem += 64 * sl;
#pragma unroll
    for (int z = SP - 1; z >= 0; --z)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            if (k0 + 16 * kt >= kw) break;
            const uint64_t da = tc::make_desc(a + (k0 / 8 + 2 * kt) * GA, GA, 128);
            const uint64_t db = TRANS ? tc::make_desc(s + z * PLANE + 256 * kt, 128, GS) : tc::make_desc(s + z * PLANE + 2 * GS * kt, GS, 128);
            tc::mma_f16(tmem, da, db, idesc, z < SP - 1 || kt > 0 || (TRANS && sl > 0));
        }
}
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[16]) {  // 16 rows x 32 columns
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// acc += f (rows r0, r0 + 8) times the warp's rows of the product at `tmem`; with DOT, returns the sums of that times the
// rows of `tile` over the columns, in every lane of the four that share them.
template <int W, bool DOT>
__device__ __forceinline__ float2 add_state(float (&acc)[W / 8][4], uint32_t tmem, float f0, float f1, const unsigned char* tile, int block,
                                            int width, int warp, int lane) {
    float s[2] = {};
    tmem += (uint32_t)(32 * (warp % 4) + 16 * (warp / 4)) << 16;
#pragma unroll
    for (int g = 0; g < W / 32; ++g) {
        if (32 * g >= width) break;
        uint32_t t[16];
        tmem_ld_rows(tmem + 32 * g, t);
        tc::tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int nt = 4 * g + u;
            if (8 * nt >= width) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = e ? f1 : f0, x = f * __uint_as_float(t[4 * u + 2 * e]), y = f * __uint_as_float(t[4 * u + 2 * e + 1]);
                acc[nt][2 * e] += x, acc[nt][2 * e + 1] += y;
                if (DOT) {
                    const uint32_t v =
                        *reinterpret_cast<const uint32_t*>(tile + nt * group_bytes(128) + (16 * place<true>(block) + lane / 4 + 8 * e) * 16 + 4 * (lane % 4));
                    s[e] = fmaf(x, lo_f(v), fmaf(y, hi_f(v), s[e]));
                }
            }
        }
    }
    if (DOT)
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
            s[1] += __shfl_xor_sync(0xffffffffu, s[1], o);
        }
    return make_float2(s[0], s[1]);
}
// A CTA's tensor memory and the barrier of its products.
struct TensorShared {
    uint64_t done, drain;
    uint32_t tmem;
    int gave_up;
};
struct Tensor {
    TensorShared& sh;
    uint32_t phase = 0;
    __device__ __forceinline__ void begin(int columns, int tid) {  // (complete after the CTA's next barrier)
        if (tid / 32 == 0) {
            tc::tmem_alloc(&sh.tmem, columns);
            tc::tmem_relinquish();
        }
        if (tid == 0) {
            tc::mbar_init(&sh.done, 1);
            tc::mbar_init(&sh.drain, 1);
            tc::mbar_fence_init();
            sh.gave_up = 0;
        }
    }
    // Every thread, before the barrier behind which one thread issues products from what this one has stored.
    static __device__ __forceinline__ void publish() {
        tc::fence_proxy_async();
        tc::fence_before_sync();
    }
    // (a wait that gives up: the results are wrong and the status word says so)
    __device__ __forceinline__ void wait() {
        if (!tc::mbar_wait_bounded(&sh.done, phase & 1, kLinattnWait)) sh.gave_up = 1;
        ++phase;
        tc::fence_after_sync();
    }
    __device__ __forceinline__ void end(int columns, int tid, unsigned* status) {
        tc::fence_before_sync();
        __syncthreads();
        if (tid == 0 && sh.gave_up) {
            tc::drain_mmas(&sh.drain, kLinattnWait);
            if (status) atomicOr(status, kStatusLinattn);
        }
        __syncwarp();
        if (tid / 32 == 0) tc::tmem_dealloc(sh.tmem, columns);
    }
};

// --------------------------------------------------------------- states
// A CTA has 64 x 64 of a state (which never mix with the others), a warp 16 rows n of them in registers, and
// takes every token's decayed key (three planes) times its value.  Tokens come 64 at a time, bfloat16 ones two
// stages ahead; the decays of eight chunks are made at once, a warp each.
template <typename E, int C>
struct StatesSmem {
    static constexpr int NP = Type<E>::NP, HT = imin(C, 64), STAGES = NP == 1 ? 3 : 2, BATCH = 8;
    static constexpr int X = NP * HT * pitch(64), Y = X;
    static constexpr int W = STAGES * (X + Y), BYTES = W + 4 * BATCH * (C + 4);
    static constexpr int THREADS = 128;
};

template <typename E, int C, bool FULL>
__global__ void __launch_bounds__(128) states_kernel(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v,
                                                        const E* __restrict__ dout, const float* __restrict__ g,
                                                        const int* __restrict__ lens, const float* h0, const float* dh_final,
                                                        float* h_final, float* gh0, Scratch w, Shape sh) {
    using M = StatesSmem<E, C>;
    constexpr int NP = M::NP, THREADS = M::THREADS, HT = M::HT, HALVES = C / HT, STAGES = M::STAGES, BATCH = M::BATCH;
    extern __shared__ __align__(128) unsigned char smem[];
    float* weights = reinterpret_cast<float*>(smem + M::W);  // [BATCH][C]
    float2* totals = reinterpret_cast<float2*>(weights + BATCH * C);  // [BATCH] a chunk's decay (exp_pair)
    delta::let_next_start();  // (the kernel behind this one waits for its end before it reads what it leaves)
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int N = sh.N, P = sh.P, s = blockIdx.y, dir = blockIdx.z;
    int slice, h;
    const int bh = sh.by_slices.div(blockIdx.x, slice), b = sh.by_h.div(bh, h), slices = (int)sh.by_slices.d;
    const int across = P > 64 ? 2 : 1, p0 = 64 * (slice % across), m0 = 64 * (slice / across), KH = sh.H / sh.G;
    const int cols = FULL ? 64 : min(64, P - p0), own = FULL ? 64 : min(64, N - m0);  // of this CTA
    const int len = row_len(lens, b, sh.T), live = (len + C - 1) / C;
    const int w0 = s * sh.seg, w1 = min(w0 + sh.seg, live);
    const int64_t np = (int64_t)N * P, row = (int64_t)dir * sh.BH + bh;
    const int n0 = 16 * warp;
    const bool mine = n0 < own, first = tid == 0 && slice == 0;
    const E* xs = (dir ? q : k) + (int64_t)(h / sh.G) * N + m0;
    const E* ys = (dir ? dout : v) + (int64_t)h * P + p0;
    const int64_t xst = (int64_t)KH * N, yst = (int64_t)sh.H * P;
    const float* gs = g + b * sh.g_row + h;
    auto chunk_of = [&](int i) { return dir ? live - 1 - i : i; };
    auto fetch = [&](int t) {  // the t-th stage of this segment
        const int i = w0 + t / HALVES, at0 = chunk_of(i) * C + t % HALVES * HT;
        if (i < w1) {
            const int64_t t0 = (int64_t)b * sh.T + min(at0, len - 1);  // (a half without tokens reads nothing)
            unsigned char* at = smem + t % STAGES * (M::X + M::Y);
            load_tile<E, 64, HT, THREADS>(at, HT * pitch(64), xs + t0 * xst, xst, len - at0, own, tid);
            load_tile<E, 64, HT, THREADS>(at + M::X, HT * pitch(64), ys + t0 * yst, yst, len - at0, cols, tid);
        }
        if (NP == 1) cp_commit();
    };
#pragma unroll
    for (int t = 0; t < STAGES - 1; ++t) fetch(t);
    float st[8][4];
    const float* start = dir ? dh_final : h0;
    auto each = [&](auto f) {  // pairs of the warp's part of the state
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int p = 8 * nt + 2 * (lane % 4);
                if (p < cols) f((int64_t)(m0 + n0 + lane / 4 + 4 * e) * P + p0 + p, st[nt][e], st[nt][e + 1]);
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
    float all = 1.f, all_lo = 0.f;  // decay since the segment's start, as two floats
    for (int i = w0, t = 0; i < w1; ++i) {
        if ((i - w0) % BATCH == 0) {
            if (i > w0) __syncthreads();  // (the weights of the batch before are read)
            for (int j = warp; j < min(BATCH, w1 - i); j += THREADS / 32) {
                const int c = chunk_of(i + j);
                const Sums<C> G = chunk_sums<C>(gs + (int64_t)c * C * sh.g_tok, sh.g_tok, len - c * C, lane);
#pragma unroll
                for (int e = 0; e < Sums<C>::K; ++e)
                    weights[j * C + Sums<C>::K * lane + e] = dir ? sh.scale * exp_of(G.G[e]) : exp_between(G.end, G.G[e]);
                if (lane == 0) totals[j] = exp_pair(G.end);
                if (dir == 0 && slice == 0) put_decays(static_cast<Decays<C>*>(w.decays)[(int64_t)bh * sh.nc + c], G, lane);
            }
            __syncthreads();
        }
        const int c = chunk_of(i);
        const float* wt = weights + (i - w0) % BATCH * C;
        const float2 total = totals[(i - w0) % BATCH];
        const bool empty = sh.nseg == 1 ? i == 0 && !start : i == w0;  // (not read by anyone)
        if (mine && !empty) {
            float* to = w.states + (row * sh.nc + c) * np;
            each([&](int64_t at, float x, float y) { *reinterpret_cast<float2*>(to + at) = make_float2(x, y); });
        }
        if (sh.nseg > 1 && first) w.dec[row * sh.nc + c] = all;
        // the leading plane's products apart from the others': small terms are not lost
        // under large ones inside the matrix instruction
        float big[8][4] = {}, rest[8][4] = {};
#pragma unroll 1
        for (int half = 0; half < HALVES; ++half, ++t) {
            if (NP == 1) cp_wait<STAGES - 2>();
            __syncthreads();
            fetch(t + STAGES - 1);
            if (!mine) continue;
            const uint32_t x = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + t % STAGES * (M::X + M::Y), y = x + M::X;
#pragma unroll
            for (int kt = 0; kt < HT / 16; ++kt) {
                uint32_t raw[NP][4], a[3][4];
#pragma unroll
                for (int z = 0; z < NP; ++z) ldsm_t(raw[z], lane_at<true>(x + z * HT * pitch(64), pitch(64), 16 * kt, n0, lane));
                const float2 u0 = *reinterpret_cast<const float2*>(wt + half * HT + 16 * kt + 2 * (lane % 4));
                const float2 u1 = *reinterpret_cast<const float2*>(wt + half * HT + 16 * kt + 8 + 2 * (lane % 4));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float e0 = lo_f(raw[NP - 1][r]), e1 = hi_f(raw[NP - 1][r]);
#pragma unroll
                    for (int z = NP - 2; z >= 0; --z) e0 += lo_f(raw[z][r]), e1 += hi_f(raw[z][r]);
                    uint32_t pl[3];
                    split<3>(e0 * (r < 2 ? u0.x : u1.x), e1 * (r < 2 ? u0.y : u1.y), pl);
                    a[0][r] = pl[0], a[1][r] = pl[1], a[2][r] = pl[2];
                }
#pragma unroll
                for (int j = NP - 1; j >= 0; --j) {
                    uint32_t bf[4][4];
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
                        if (16 * nt < cols) ldsm_t(bf[nt], lane_at<false>(y + j * HT * pitch(64), pitch(64), 16 * kt, 16 * nt, lane));
#pragma unroll
                    for (int z = 2; z >= 0; --z)
                        if (z + j < 3)
#pragma unroll
                            for (int nt = 0; nt < 4; ++nt)
                                if (16 * nt < cols) {
                                    float(&c0)[4] = z + j == 0 ? big[2 * nt] : rest[2 * nt];
                                    float(&c1)[4] = z + j == 0 ? big[2 * nt + 1] : rest[2 * nt + 1];
                                    mma(c0, a[z], bf[nt][0], bf[nt][1]);
                                    mma(c1, a[z], bf[nt][2], bf[nt][3]);
                                }
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) st[nt][e] = fmaf(total.x, st[nt][e], fmaf(total.y, st[nt][e], big[nt][e] + rest[nt][e]));
        const float p = all * total.x, left = fmaf(all, total.x, -p) + fmaf(all, total.y, all_lo * total.x);
        all = p + left;
        all_lo = left - (all - p);
    }
    float* last = dir ? gh0 : h_final;
    if (sh.nseg == 1) {
        if (mine && last)
            each([&](int64_t at, float x, float y) { *reinterpret_cast<float2*>(last + bh * np + at) = make_float2(x, y); });
        return;
    }
    // the segments' own states at their ends, from which each makes the state before it
    float* ends = w.ends + row * sh.nseg * np;
    if (mine) each([&](int64_t at, float x, float y) { *reinterpret_cast<float2*>(ends + s * np + at) = make_float2(x, y); });
    if (tid == 0) w.seg_all[(row * slices + slice) * sh.nseg + s] = all;
    auto cluster_sync = [] { asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory"); };
    cluster_sync();
    if (mine) {
        const float* alls = w.seg_all + (row * slices + slice) * sh.nseg;
        float r[8][4] = {};  // the state before this segment: from the nearest one back
        auto add = [&](const float* from, float d) {  // (all loads before the sums)
            float2 a[16];
            int i = 0;
            each([&](int64_t at, float&, float&) { a[i++] = __ldcg(reinterpret_cast<const float2*>(from + at)); });
            i = 0;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; e += 2)
                    if (8 * nt + 2 * (lane % 4) < cols) {
                        r[nt][e] = fmaf(d, a[i].x, r[nt][e]), r[nt][e + 1] = fmaf(d, a[i].y, r[nt][e + 1]);
                        ++i;
                    }
        };
        float d = 1.f;
        for (int e = s - 1; e >= 0; --e) {
            add(ends + e * np, d);
            d *= __ldcg(alls + e);
        }
        if (start) add(start + bh * np, d);
        if (s > 0 || start) {
            float* to = w.starts + (row * sh.nseg + s) * np;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int p = 8 * nt + 2 * (lane % 4);
                    if (p < cols)
                        *reinterpret_cast<float2*>(to + (int64_t)(m0 + n0 + lane / 4 + 4 * e) * P + p0 + p) = make_float2(r[nt][e], r[nt][e + 1]);
                }
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) st[nt][e] = fmaf(all, r[nt][e], st[nt][e]);
    }
    if (!last) return;
    if (start) cluster_sync();  // (the last state may lie over the first)
    if (mine && s == max((live + sh.seg - 1) / sh.seg - 1, 0))  // the row's last segment
        each([&](int64_t at, float x, float y) { *reinterpret_cast<float2*>(last + bh * np + at) = make_float2(x, y); });
}

// --------------------------------------------------------------- outputs
// A warp's 16 rows and CW columns (from col0) of `acc`, times `factor`, to tokens of a tensor with `stride` elements
// between them: n rows have values, those from n to `rows` are zeros.  16-bit types go through `stage` (the
// warp's 16 rows, OW columns) for whole 16-byte stores.
template <typename E, int OW, int CW>
__device__ __forceinline__ void put_rows(E* out, int64_t stride, const float (&acc)[CW / 8][4], float factor, unsigned char* stage, int col0,
                                         int ow, int n, int rows, int lane) {
    if constexpr (sizeof(E) == 2) {
        unsigned char* at = stage + lane / 4 * pitch(OW) + 2 * col0 + 4 * (lane % 4);
        __syncwarp();  // (what was staged here before is read)
#pragma unroll
        for (int nt = 0; nt < CW / 8; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                alignas(4) E w[2] = {from_f<E>(factor * acc[nt][2 * e]), from_f<E>(factor * acc[nt][2 * e + 1])};
                *reinterpret_cast<uint32_t*>(at + 8 * e * pitch(OW) + 16 * nt) = *reinterpret_cast<uint32_t*>(w);
            }
        __syncwarp();
        constexpr int PER = CW / 8, STEP = 32 / PER;
        const int c = col0 + lane % PER * 8;
#pragma unroll
        for (int r0 = 0; r0 < 16; r0 += STEP) {
            const int r = r0 + lane / PER;
            if (r < rows && c < ow)
                __stcs(reinterpret_cast<uint4*>(out + r * stride + c),
                       r < n ? *reinterpret_cast<const uint4*>(stage + r * pitch(OW) + 2 * c) : make_uint4(0, 0, 0, 0));
        }
    } else {
#pragma unroll
        for (int nt = 0; nt < CW / 8; ++nt) {
            if (col0 + 8 * nt >= ow) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = lane / 4 + 8 * e;
                if (r < rows)
                    *reinterpret_cast<float2*>(out + r * stride + col0 + 8 * nt + 2 * (lane % 4)) =
                        r < n ? make_float2(factor * acc[nt][2 * e], factor * acc[nt][2 * e + 1]) : make_float2(0.f, 0.f);
            }
        }
    }
}
// Zeros over `rows` tokens of a chunk that has none.
template <typename E>
__device__ __forceinline__ void clear_rows(E* at, int64_t stride, int width, int rows, int tid) {
    const int per = width * (int)sizeof(E) / 16;
    for (int i = tid; i < rows * per; i += NT) reinterpret_cast<uint4*>(at + (i / per) * stride)[i % per] = make_uint4(0, 0, 0, 0);
}
// The first `bytes` of a chunk's tables, by cp.async.
__device__ __forceinline__ void load_decays(unsigned char* dst, const void* src, int bytes, int tid) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    for (int i = tid; i < bytes / 16; i += NT) cp16(to + 16 * i, static_cast<const unsigned char*>(src) + 16 * i, true);
}

// Three CTAs an SM at 64/64 (80 registers, 76 KB): 37 us for 4 x 2048 x 24, tensor pipe 42 % busy, issue 38 %; with
// two blocks of scores in flight a warp at two CTAs an SM the call took 71.0 us against 68.9.
template <typename E, int ND, int PD, int C>
struct OutSmem {
    static constexpr int NP = Type<E>::NP, SP = NP == 3 ? 3 : 2;
    static constexpr int X = NP * Tile<false, C, ND>::PLANE, Y = NP * Tile<false, C, PD>::PLANE;
    static constexpr int Q = 0, K = X, V = 2 * X, S = 2 * X + Y;
    static constexpr int D = S + imax(SP * Tile<false, 64, PD>::PLANE, sizeof(E) == 2 ? C * pitch(PD) : 0);
    static constexpr int TABLE = sizeof(Decays<C>) - 4 * C, BYTES = D + TABLE;
    static constexpr int CTAS = BYTES + 1024 <= 76 * 1024 ? 3 : BYTES + 1024 <= 114 * 1024 ? 2 : 1;
};

template <typename E, int ND, int PD, int C, bool FULL>
__global__ void __launch_bounds__(NT, OutSmem<E, ND, PD, C>::CTAS)
    out_kernel(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v, const int* __restrict__ lens, bool start,
               E* __restrict__ o, Scratch w, Shape sh) {
    using M = OutSmem<E, ND, PD, C>;
    constexpr int NP = M::NP, SP = M::SP, CW = PD / Part<C>::CS;
    extern __shared__ __align__(128) unsigned char smem[];
    const Decays<C>& d = *reinterpret_cast<const Decays<C>*>(smem + M::D);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int N = FULL ? ND : sh.N, P = FULL ? PD : sh.P, KH = sh.H / sh.G;
    int h, c;
    const int b = sh.by_nc.div(sh.by_h.div(blockIdx.x, h), c);
    const int len = row_len(lens, b, sh.T), live = (len + C - 1) / C, n = min(len - c * C, C), rows = min(sh.T - c * C, C);
    const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C, bh = (int64_t)b * sh.H + h, os = (int64_t)sh.H * P;
    E* orow = o + t0 * os + (int64_t)h * P;
    if (n <= 0) {
        delta::wait_for_previous();  // (no block writes or ends before the kernel before this one has)
        return clear_rows(orow, os, P, rows, tid);
    }
    const int64_t ks = (int64_t)KH * N, ko = t0 * ks + (int64_t)(h / sh.G) * N;
    load_tile<E, ND, C, NT>(smem + M::Q, C * pitch(ND), q + ko, ks, n, N, tid);
    load_tile<E, ND, C, NT>(smem + M::K, C * pitch(ND), k + ko, ks, n, N, tid);
    load_tile<E, PD, C, NT>(smem + M::V, C * pitch(PD), v + t0 * os + (int64_t)h * P, os, n, P, tid);
    delta::wait_for_previous();  // (from here on: what the states' walk left)
    load_decays(smem + M::D, static_cast<const Decays<C>*>(w.decays) + bh * sh.nc + c, M::TABLE, tid);
    cp_commit();
    const StateAt st = state_at(w, sh, 0, bh, c, live, start);
    StateTile<SP, PD, false> tile;
    if (st.any()) {
        tile.fetch(st, 0, N, P, tid);
        tile.put(smem + M::S, tid);
    }
    cp_wait<0>();
    __syncthreads();
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const Part<C> part(warp);
    const int block = part.block, col0 = part.share * CW, r0 = 16 * block + lane / 4;
    float acc[CW / 8][4] = {};
    if (st.any()) {
#pragma unroll
        for (int sl = 0; sl < ND / 64; ++sl) {
            if (64 * sl >= N) break;
            if (sl) {
                tile.fetch(st, sl, N, P, tid);
                __syncthreads();
                tile.put(smem + M::S, tid);
                __syncthreads();
            }
            times_state<NP, SP, C, ND, PD, CW, true>(acc, base + M::Q, base + M::S, block, col0, sl, N, P, lane);
        }
        scale_rows(acc, d.in[r0], d.in[r0 + 8]);
    }
    if (16 * block < n)
        earlier_pairs<NP, NP, SP, C, ND, PD, CW, false>(acc, base + M::Q, base + M::K, base + M::V, block, col0, N, P, 1.f, d, lane);
    if (sizeof(E) == 2 && st.any()) __syncthreads();  // (the state's planes are read: the stage lies over them)
    put_rows<E, PD, CW>(orow + 16 * block * os, os, acc, sh.scale, smem + M::S + 16 * block * pitch(PD), col0, P, n - 16 * block,
                        rows - 16 * block, lane);
}

// --------------------------------------------------------------- gradients
// 4 x 2048 x 24, 64/64: 139 us at two CTAs an SM, tensor pipe 37 % busy, issue 33 % (dk and dv 50 us, the state's
// products 45, dq 15, loads and stores the rest).  128/128: one CTA an SM (four tiles of 34 KB), 255 registers; there
// the state's products by the warps were half of it (80 of 157 us), whose operands' reads from shared memory (2 MB a
// chunk) and tensor time (27000 cycles a chunk) were equal, so they are tcgen05 ones beside the scores.  16 warps a
// CTA, sharing columns, took 225 us a call against 212 there (without tcgen05) and 256 against 184 at 64/64 (scores twice).
// The states have three planes for dq and dk, from which dg (a float32 result) takes its terms, and two for dv.
template <typename E, int ND, int PD, int C>
struct GradSmem {
    static constexpr int NP = Type<E>::NP, SP = NP == 3 ? 3 : 2, RB = C / 16;
    // The state's products on tcgen05 for the wide tiles: 195 us against 216 for 4 x 1501 x 16 on 8 key heads, 128/128;
    // at 64/64, where two CTAs an SM leave 128 registers a thread, 188 against 184 for 4 x 2048 x 24.
    static constexpr bool TC = C == 128 && (ND > 64 || PD > 64);
    static constexpr int X = NP * Tile<TC, C, ND>::PLANE, Y = NP * Tile<TC, C, PD>::PLANE;
    static constexpr int Q = 0, K = X, V = 2 * X, DO = 2 * X + Y, S = 2 * X + 2 * Y;
    static constexpr int D = S + imax(3 * Tile<TC, 64, PD>::PLANE, sizeof(E) == 2 ? C * pitch(imax(ND, PD)) : 0);
    static constexpr int COLUMNS = ND + PD == 192 ? 256 : ND + PD;  // of tensor memory: dq, then dk; dv
    static constexpr int COL = D + sizeof(Decays<C>);      // [RB][C] sums of W over the tokens j of a block
    static constexpr int ROW = COL + 4 * RB * C;           // [C] sums of W over i
    static constexpr int AQ = ROW + 4 * C, BK = AQ + 8 / RB * C * 4, BYTES = BK + 8 / RB * C * 4;  // [share][C]
    static constexpr int CTAS = BYTES + 1280 <= 114 * 1024 ? 2 : 1;
};

// Sum over a row's columns of the accumulators times a tile's values (rows r0 and r0 + 8), in every lane of the
// four that share the rows.
template <int NPL, int C, int W, int CW>
__device__ __forceinline__ float2 dot_rows(const float (&acc)[CW / 8][4], const unsigned char* tile, int block, int col0, int width, int lane) {
    float s[2] = {};
    const unsigned char* at = tile + (16 * block + lane / 4) * pitch(W) + 2 * col0 + 4 * (lane % 4);
#pragma unroll
    for (int nt = 0; nt < CW / 8; ++nt) {
        if (col0 + 8 * nt >= width) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int z = NPL - 1; z >= 0; --z) {
                const uint32_t v = *reinterpret_cast<const uint32_t*>(at + z * C * pitch(W) + 8 * e * pitch(W) + 16 * nt);
                x += lo_f(v), y += hi_f(v);
            }
            s[e] = fmaf(acc[nt][2 * e], x, fmaf(acc[nt][2 * e + 1], y, s[e]));
        }
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
        s[1] += __shfl_xor_sync(0xffffffffu, s[1], o);
    }
    return make_float2(s[0], s[1]);
}

template <typename E, int ND, int PD, int C, bool FULL>
__global__ void __launch_bounds__(NT, GradSmem<E, ND, PD, C>::CTAS)
    grad_kernel(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v, const E* __restrict__ dout,
                const int* __restrict__ lens, bool start, bool end, E* __restrict__ gq, E* __restrict__ gk, E* __restrict__ gv,
                float* __restrict__ parts, float* __restrict__ gg, float* __restrict__ gg_part, Scratch w, Shape sh, unsigned* status) {
    using M = GradSmem<E, ND, PD, C>;
    constexpr int NP = M::NP, SP = M::SP, QP = NP == 1 ? 1 : 3, CN = ND / Part<C>::CS, CP = PD / Part<C>::CS, SHARES = Part<C>::CS;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_dot[NT / 32];
    __shared__ __align__(16) TensorShared tensor_sh;
    Tensor tensor{tensor_sh};
    const Decays<C>& d = *reinterpret_cast<const Decays<C>*>(smem + M::D);
    float(*s_col)[C] = reinterpret_cast<float(*)[C]>(smem + M::COL);
    float* s_row = reinterpret_cast<float*>(smem + M::ROW);
    float(*s_aq)[C] = reinterpret_cast<float(*)[C]>(smem + M::AQ);
    float(*s_bk)[C] = reinterpret_cast<float(*)[C]>(smem + M::BK);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int N = FULL ? ND : sh.N, P = FULL ? PD : sh.P, KH = sh.H / sh.G;
    int h, c;
    const int b = sh.by_nc.div(sh.by_h.div(blockIdx.x, h), c);
    const int len = row_len(lens, b, sh.T), live = (len + C - 1) / C, n = min(len - c * C, C), rows = min(sh.T - c * C, C);
    const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C, bh = (int64_t)b * sh.H + h;
    const int64_t ks = (int64_t)KH * N, ko = t0 * ks + (int64_t)(h / sh.G) * N;
    const int64_t os = (int64_t)sh.H * P, oo = t0 * os + (int64_t)h * P;
    // with shared key heads a value head leaves its part in fp32
    const int64_t ps = (int64_t)sh.H * N, po = t0 * ps + (int64_t)h * N, pk = (int64_t)(gridDim.x / (sh.nc * sh.H)) * sh.T * ps;
    float* ggp = gg ? gg + t0 * sh.H + h : nullptr;
    if (n <= 0) {
        delta::wait_for_previous();  // (no block writes or ends before the kernel before this one has)
        clear_rows(gv + oo, os, P, rows, tid);
        if (parts) {
            clear_rows(parts + po, ps, N, rows, tid);
            clear_rows(parts + pk + po, ps, N, rows, tid);
        } else {
            clear_rows(gq + ko, ks, N, rows, tid);
            clear_rows(gk + ko, ks, N, rows, tid);
        }
        if (ggp)
            for (int i = tid; i < rows; i += NT) ggp[(int64_t)i * sh.H] = 0.f;
        if (gg_part && tid == 0) gg_part[blockIdx.x] = 0.f;
        return;
    }
    if (M::TC) tensor.begin(M::COLUMNS, tid);
    auto load = [&](auto width, unsigned char* to, const E* from, int64_t stride, int tokens, int columns) {
        constexpr int W = decltype(width)::value;
        if constexpr (M::TC)
            load_core<W, NT>(to, from, stride, tokens, columns, tid);
        else
            load_tile<E, W, C, NT>(to, C * pitch(W), from, stride, tokens, columns, tid);
    };
    load(std::integral_constant<int, PD>(), smem + M::DO, dout + oo, os, n, P);
    load(std::integral_constant<int, PD>(), smem + M::V, v + oo, os, n, P);
    load(std::integral_constant<int, ND>(), smem + M::K, k + ko, ks, n, N);
    load(std::integral_constant<int, ND>(), smem + M::Q, q + ko, ks, n, N);
    delta::wait_for_previous();  // (from here on: what the states' walk left)
    load_decays(smem + M::D, static_cast<const Decays<C>*>(w.decays) + bh * sh.nc + c, sizeof(Decays<C>), tid);
    cp_commit();
    const StateAt sb = state_at(w, sh, 0, bh, c, live, start), sa = state_at(w, sh, 1, bh, c, live, end);
    StateTile<3, PD, M::TC> tile;
    if (sb.any()) {
        tile.fetch(sb, 0, N, P, tid);
        tile.put(smem + M::S, tid);
    }
    cp_wait<0>();
    if (M::TC) Tensor::publish();
    __syncthreads();
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const Part<C> part(warp);
    const int block = part.block, r0 = 16 * block + lane / 4, last = (n + 15) / 16, nq = 16 * block;
    const int colN = part.share * CN, colP = part.share * CP;
    const bool on = block < last;
    const float scale = sh.scale;
    {
        float acc[CN / 8][4] = {};
        float2 a = make_float2(0.f, 0.f);
        if (sb.any()) {
#pragma unroll
            for (int sl = 0; sl < ND / 64; ++sl) {
                if (64 * sl >= N) break;
                if (sl) {
                    tile.fetch(sb, sl, N, P, tid);
                    if (M::TC) tensor.wait();
                    __syncthreads();
                    tile.put(smem + M::S, tid);
                    if (M::TC) Tensor::publish();
                    __syncthreads();
                }
                if constexpr (M::TC) {
                    if (tid == 0) {
                        tc::fence_after_sync();
                        issue_state<PD, ND, 3, false>(tensor_sh.tmem, base + M::DO, base + M::S, sl, P);
                        tc::commit(&tensor_sh.done);
                    }
                    __syncwarp();
                } else {
                    times_state<NP, 3, C, PD, ND, CN, false>(acc, base + M::DO, base + M::S, block, colN, sl, P, N, lane);
                }
            }
            if (!M::TC) {
                scale_rows(acc, scale * d.in[r0], scale * d.in[r0 + 8]);
                a = dot_rows<NP, C, ND, CN>(acc, smem + M::Q, block, colN, N, lane);
            }
        }
        if (on) earlier_pairs<NP, QP, SP, C, PD, ND, CN, M::TC>(acc, base + M::DO, base + M::V, base + M::K, block, colN, P, N, scale, d, lane);
        if constexpr (M::TC) {
            if (sb.any()) {
                tensor.wait();
                a = add_state<ND, true>(acc, tensor_sh.tmem, scale * d.in[r0], scale * d.in[r0 + 8], smem + M::Q, block, N, warp, lane);
                tc::fence_before_sync();  // (dk's product comes over this one behind the next barrier)
            }
        } else if (sizeof(E) == 2 && sb.any()) {
            __syncthreads();  // (the stage lies over the state's planes)
        }
        if (lane % 4 == 0) s_aq[part.share][r0] = a.x, s_aq[part.share][r0 + 8] = a.y;
        if (parts)
            put_rows<float, ND, CN>(parts + po + nq * ps, ps, acc, 1.f, nullptr, colN, N, n - nq, rows - nq, lane);
        else
            put_rows<E, ND, CN>(gq + ko + nq * ks, ks, acc, 1.f, smem + M::S + nq * pitch(ND), colN, N, n - nq, rows - nq, lane);
    }
    float dot = 0.f;  // <S, dS+>
    float dk[CN / 8][4] = {}, dv[CP / 8][4] = {};
    float2 own = make_float2(0.f, 0.f);
    if (sa.any()) {
        const bool both = sb.any();
#pragma unroll
        for (int sl = 0; sl < ND / 64; ++sl) {
            if (64 * sl >= N) break;
            tile.fetch(sa, sl, N, P, tid);
            if (M::TC && sl) tensor.wait();
            __syncthreads();
            tile.put(smem + M::S, tid);
            if (both) {
                using ST = StateTile<3, PD, M::TC>;
                const int r = 64 * sl + tid / ST::PER, x = 4 * (tid % ST::PER);
#pragma unroll
                for (int e = 0; e < ST::K; ++e)
                    if (x < P && r + ST::STEP * e < N) {
                        const float4 u = sb.at((r + ST::STEP * e) * P + x), y = tile.v[e];
                        dot = fmaf(u.x, y.x, fmaf(u.y, y.y, fmaf(u.z, y.z, fmaf(u.w, y.w, dot))));
                    }
            }
            if (M::TC) Tensor::publish();
            __syncthreads();
            if constexpr (M::TC) {
                if (tid == 0) {
                    tc::fence_after_sync();
                    issue_state<PD, ND, 3, false>(tensor_sh.tmem, base + M::V, base + M::S, sl, P);
                    issue_state<ND, PD, SP, true>(tensor_sh.tmem + ND, base + M::K, base + M::S, sl, N);
                    tc::commit(&tensor_sh.done);
                }
                __syncwarp();
            } else {
                times_state<NP, 3, C, PD, ND, CN, false>(dk, base + M::V, base + M::S, block, colN, sl, P, N, lane);
                times_state<NP, SP, C, ND, PD, CP, true>(dv, base + M::K, base + M::S, block, colP, sl, N, P, lane);
            }
        }
        if (!M::TC) {
            scale_rows(dk, d.out[r0], d.out[r0 + 8]);
            scale_rows(dv, d.out[r0], d.out[r0 + 8]);
            own = dot_rows<NP, C, ND, CN>(dk, smem + M::K, block, colN, N, lane);
        }
    }
    float wr[2] = {};  // sums of W over the tokens i
    if (on) {
        const Rows<NP, C, ND, M::TC> rk(base + M::K, block, N, lane);
        const Rows<NP, C, PD, M::TC> rv(base + M::V, block, P, lane);
        float row[2];
        row_factors<C, false>(row, d, block, scale, lane);
#pragma unroll 1
        for (int o = block; o < last; ++o) {
            float sa_[2][4], sb_[2][4], m[2][4];
            scores<NP, QP, C, ND, M::TC>(sa_, rk, base + M::Q, o, N, lane);   // k_j . q_i
            scores<NP, QP, C, PD, M::TC>(sb_, rv, base + M::DO, o, P, lane);  // v_j . do_i
            if (o != block) {
                pair_factors<C, false, false>(m, d, block, o, row, scale, lane);
            } else {
                pair_factors<C, false, true>(m, d, block, o, row, scale, lane);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (8 * x + 2 * (lane % 4) + e % 2 < lane / 4 + 8 * (e / 2)) sa_[x][e] = sb_[x][e] = 0.f;
            }
            multiply(sa_, m);
            float ws[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) ws[x][e] = sa_[x][e] * sb_[x][e];
            if (o == block) {  // (a token's own write spans no decay)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 2 * x; e < 2 * x + 2; ++e)
                        if (2 * (lane % 4) + e % 2 == lane / 4) ws[x][e] = 0.f;
            }
            multiply(sb_, m);
            wr[0] += (ws[0][0] + ws[0][1]) + (ws[1][0] + ws[1][1]);
            wr[1] += (ws[0][2] + ws[0][3]) + (ws[1][2] + ws[1][3]);
            {  // over the 16 tokens j, for the four columns of a lane: halves change hands
                float c0 = ws[0][0] + ws[0][2], c1 = ws[0][1] + ws[0][3], c2 = ws[1][0] + ws[1][2], c3 = ws[1][1] + ws[1][3];
                const bool up = lane & 16, odd = lane & 8;
                const float g0 = __shfl_xor_sync(0xffffffffu, up ? c0 : c2, 16), g1 = __shfl_xor_sync(0xffffffffu, up ? c1 : c3, 16);
                c0 = (up ? c2 : c0) + g0, c1 = (up ? c3 : c1) + g1;
                const float g2 = __shfl_xor_sync(0xffffffffu, odd ? c0 : c1, 8);
                c0 = (odd ? c1 : c0) + g2;
                c0 += __shfl_xor_sync(0xffffffffu, c0, 4);
                if (!(lane & 4) && part.share == 0) s_col[block][16 * o + (up ? 8 : 0) + 2 * (lane % 4) + (odd ? 1 : 0)] = c0;
            }
            times_tokens<NP, SP, C, PD, CP, M::TC>(dv, sa_, base + M::DO, colP, o, P, lane);
            times_tokens<NP, SP, C, ND, CN, M::TC>(dk, sb_, base + M::Q, colN, o, N, lane);
        }
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        wr[0] += __shfl_xor_sync(0xffffffffu, wr[0], o);
        wr[1] += __shfl_xor_sync(0xffffffffu, wr[1], o);
    }
    if constexpr (M::TC)
        if (sa.any()) {
            tensor.wait();
            own = add_state<ND, true>(dk, tensor_sh.tmem, d.out[r0], d.out[r0 + 8], smem + M::K, block, N, warp, lane);
            add_state<PD, false>(dv, tensor_sh.tmem + ND, d.out[r0], d.out[r0 + 8], nullptr, block, P, warp, lane);
        }
    if (lane % 4 == 0) s_bk[part.share][r0] = own.x, s_bk[part.share][r0 + 8] = own.y;
    if (lane % 4 == 0 && part.share == 0) s_row[r0] = wr[0], s_row[r0 + 8] = wr[1];
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_dot[warp] = dot;
    __syncthreads();
    if (parts)
        put_rows<float, ND, CN>(parts + pk + po + nq * ps, ps, dk, 1.f, nullptr, colN, N, n - nq, rows - nq, lane);
    else
        put_rows<E, ND, CN>(gk + ko + nq * ks, ks, dk, 1.f, smem + M::S + nq * pitch(ND), colN, N, n - nq, rows - nq, lane);
    if (sizeof(E) == 2 && (ND != PD || !parts)) __syncthreads();  // (the stage's rows lie elsewhere now, or are still read)
    put_rows<E, PD, CP>(gv + oo + nq * os, os, dv, 1.f, smem + M::S + nq * pitch(PD), colP, P, n - nq, rows - nq, lane);
    if (warp == 0 && (ggp || gg_part)) {
        float all = 0.f;
        for (int i = 0; i < NT / 32; ++i) all += s_dot[i];
        all *= d.all;
        constexpr int PER = C / 32;
        float r[PER], bk[PER], tail = 0.f, head = 0.f;  // suffix sums of a lane's tokens, and prefix sums before each
#pragma unroll
        for (int e = PER - 1; e >= 0; --e) {
            const int i = PER * lane + e;
            float x = 0.f;
            if (i < 16 * last) {
#pragma unroll
                for (int u = 0; u < SHARES; ++u) x += s_aq[u][i];
                float y = 0.f;
                for (int u = 0; u <= i / 16; ++u) y += s_col[u][i];
                x += y - s_row[i];
            }
            tail += x;
            r[e] = tail;
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            bk[e] = head;
#pragma unroll
            for (int u = 0; u < SHARES; ++u) head += s_bk[u][PER * lane + e];
        }
        float after = tail, before = head;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, after, o), y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane + o < 32) after += x;
            if (lane >= o) before += y;
        }
        after = __shfl_down_sync(0xffffffffu, after, 1);
        before = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 31) after = 0.f;
        if (lane == 0) before = 0.f;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int i = PER * lane + e;
            const float x = i < n ? all + (before + bk[e]) + (after + r[e]) : 0.f;
            sum += x;
            if (ggp && i < rows) ggp[(int64_t)i * sh.H] = x;
        }
        if (gg_part) {
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) gg_part[blockIdx.x] = sum;
        }
    }
    if (M::TC) tensor.end(M::COLUMNS, tid, status);
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
// The chunk: what leaves a chunk's tiles of the gradients and 64 rows of a state room in one SM's shared memory.
template <typename E, int ND, int PD>
constexpr int chunk_tokens() {
    return Type<E>::NP == 1 ? 128 : Type<E>::NP == 2 ? 64 : imax(ND, PD) == 64 ? 64 : 32;
}
inline int chunk_of(const LinattnArgs& a) {
    if (a.dtype == CSSD_BF16) return 128;
    if (a.dtype == CSSD_F16) return 64;
    return a.N <= 64 && a.P <= 64 ? 64 : 32;
}
inline size_t decays_bytes(const LinattnArgs& a) {
    const int C = chunk_of(a);
    return C == 128 ? sizeof(Decays<128>) : C == 64 ? sizeof(Decays<64>) : sizeof(Decays<32>);
}

// CTAs that the states' walk may have, by cutting rows into segments: as many as are resident at once where clusters
// of segments have to fit a group of SMs (1 x 16384 x 32, 128/64: 299 us with 6 segments a row, 331 with 7, 307 with 4;
// 4 x 2048 x 24, 64/64: 68.9 with 4, 69.6 with 3, 75.0 with 2; its gradients 189 with 2, 193 uncut).
constexpr int kStateCtas = 384;
inline int slices_of(const LinattnArgs& a) { return (a.N > 64 ? 2 : 1) * (a.P > 64 ? 2 : 1); }

inline Shape shape_of(const LinattnArgs& a, int dirs) {
    Shape sh{};
    const int C = chunk_of(a);
    sh.T = (int)a.T, sh.H = (int)a.H, sh.G = (int)(a.H / a.KH), sh.N = (int)a.N, sh.P = (int)a.P;
    sh.nc = (int)((a.T + C - 1) / C);
    sh.BH = (int)(a.Bz * a.H);
    const int64_t rows = a.Bz * a.H * dirs * slices_of(a);
    int64_t want = rows >= kStateCtas ? 1 : kStateCtas / rows;
    if (want > kMostSegments) want = kMostSegments;
    sh.seg = (int)((sh.nc + want - 1) / want);
    sh.nseg = (sh.nc + sh.seg - 1) / sh.seg;
    sh.g_row = a.g_tokens ? a.T * a.H : 0;
    sh.g_tok = a.g_tokens ? a.H : 0;
    sh.scale = a.scale;
    sh.by_h = Divisor::of((uint32_t)sh.H);
    sh.by_nc = Divisor::of((uint32_t)sh.nc);
    sh.by_slices = Divisor::of((uint32_t)slices_of(a));
    return sh;
}

inline size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

// The workspace's parts; returns what they take together.
inline size_t scratch_of(const LinattnArgs& a, int dirs, void* ws, Scratch& s) {
    const Shape sh = shape_of(a, dirs);
    const size_t rows = (size_t)dirs * sh.BH, np = (size_t)sh.N * sh.P * 4;
    size_t at = 0;
    auto take = [&](size_t n) {
        void* p = static_cast<unsigned char*>(ws) + at;
        at += up(n);
        return static_cast<float*>(p);
    };
    s = Scratch{};
    s.states = take(rows * sh.nc * np);
    s.decays = take((size_t)sh.BH * sh.nc * decays_bytes(a));
    if (sh.nseg > 1) {
        s.ends = take(rows * sh.nseg * np);
        s.starts = take(rows * sh.nseg * np);
        s.seg_all = take(rows * slices_of(a) * sh.nseg * 4);
        s.dec = take(rows * sh.nc * 4);
    }
    return at;
}
inline size_t scratch_bytes(const LinattnArgs& a, int dirs) {
    Scratch s;
    return scratch_of(a, dirs, nullptr, s);
}

template <typename E, int C, bool FULL>
cudaError_t run_states(const LinattnArgs& a, int dirs, const Scratch& w, const Shape& sh, cudaStream_t st) {
    using M = StatesSmem<E, C>;
    cudaError_t e = delta::allow<states_kernel<E, C, FULL>>(M::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.BH * slices_of(a), sh.nseg, dirs);
    cfg.blockDim = dim3(M::THREADS);
    cfg.dynamicSmemBytes = M::BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1, attr.val.clusterDim.y = sh.nseg, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, states_kernel<E, C, FULL>, static_cast<const E*>(a.q), static_cast<const E*>(a.k),
                              static_cast<const E*>(a.v), static_cast<const E*>(a.dout), a.g, a.lens, a.h0, a.dh_final, a.h_final, a.gh0, w,
                              sh);
}

// Launches a kernel that may start while the one before it in the stream still runs.
template <typename... A, typename... B>
cudaError_t launch_behind(void (*kernel)(A...), unsigned grid, int bytes, cudaStream_t st, B... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<A>(args)...);
}

template <typename E, int ND, int PD, bool FULL>
cudaError_t forward(const LinattnArgs& a, void* ws, cudaStream_t st) {
    constexpr int C = chunk_tokens<E, ND, PD>();
    using M = OutSmem<E, ND, PD, C>;
    const Shape sh = shape_of(a, 1);
    Scratch w;
    scratch_of(a, 1, ws, w);
    cudaError_t e = run_states<E, C, FULL>(a, 1, w, sh, st);
    if (e == cudaSuccess) e = delta::allow<out_kernel<E, ND, PD, C, FULL>>(M::BYTES);
    if (e != cudaSuccess) return e;
    return launch_behind(out_kernel<E, ND, PD, C, FULL>, (unsigned)(sh.BH * sh.nc), M::BYTES, st, static_cast<const E*>(a.q),
                         static_cast<const E*>(a.k), static_cast<const E*>(a.v), a.lens, a.h0 != nullptr, static_cast<E*>(a.o), w, sh);
}

inline size_t parts_bytes(const LinattnArgs& a) { return a.H == a.KH ? 0 : up((size_t)2 * a.Bz * a.T * a.H * a.N * 4); }

template <typename E, int ND, int PD, bool FULL>
cudaError_t backward(const LinattnArgs& a, void* ws, cudaStream_t st) {
    constexpr int C = chunk_tokens<E, ND, PD>();
    using M = GradSmem<E, ND, PD, C>;
    const Shape sh = shape_of(a, 2);
    Scratch w;
    unsigned char* rest = static_cast<unsigned char*>(ws) + scratch_of(a, 2, ws, w);
    float* parts = parts_bytes(a) ? reinterpret_cast<float*>(rest) : nullptr;
    float* gg_part = a.gg && !a.g_tokens ? reinterpret_cast<float*>(rest + parts_bytes(a)) : nullptr;
    cudaError_t e = run_states<E, C, FULL>(a, 2, w, sh, st);
    if (e == cudaSuccess) e = delta::allow<grad_kernel<E, ND, PD, C, FULL>>(M::BYTES);
    if (e != cudaSuccess) return e;
    e = launch_behind(grad_kernel<E, ND, PD, C, FULL>, (unsigned)(sh.BH * sh.nc), M::BYTES, st, static_cast<const E*>(a.q),
                      static_cast<const E*>(a.k), static_cast<const E*>(a.v), static_cast<const E*>(a.dout), a.lens, a.h0 != nullptr,
                      a.dh_final != nullptr, static_cast<E*>(a.gq), static_cast<E*>(a.gk), static_cast<E*>(a.gv), parts,
                      a.g_tokens ? a.gg : nullptr, gg_part, w, sh, status_word());
    if (e != cudaSuccess) return e;
    if (parts) {
        const int64_t vectors = a.Bz * a.T * a.KH * (a.N / 4);
        join_kernel<E><<<dim3((unsigned)((vectors + 255) / 256), 2), 256, 0, st>>>(parts, static_cast<E*>(a.gq), static_cast<E*>(a.gk),
                                                                                  vectors, a.Bz * a.T * a.H * a.N, sh.G, sh.N);
    }
    if (gg_part) join_g_kernel<<<sh.H, 128, 0, st>>>(gg_part, a.gg, a.Bz * sh.nc, sh.H);
    return cudaGetLastError();
}

// Calls f with the widths' tiles (64 or 128 columns) and whether the widths fill them: the kernels then have no
// tests of columns (4 x 2048 x 24, 64/64: forward 75 us against 87, gradients 194 against 244).
template <typename F>
cudaError_t by_widths(const LinattnArgs& a, F f) {
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    auto full = [&](auto n, auto p) {
        return a.N == decltype(n)::value && a.P == decltype(p)::value ? f(n, p, std::true_type()) : f(n, p, std::false_type());
    };
    if (a.N <= 64) return a.P <= 64 ? full(I64(), I64()) : full(I64(), I128());
    return a.P <= 64 ? full(I128(), I64()) : full(I128(), I128());
}
template <typename E>
cudaError_t forward_of(const LinattnArgs& a, void* ws, cudaStream_t st) {
    return by_widths(a, [&](auto n, auto p, auto full) {
        return forward<E, decltype(n)::value, decltype(p)::value, decltype(full)::value>(a, ws, st);
    });
}
template <typename E>
cudaError_t backward_of(const LinattnArgs& a, void* ws, cudaStream_t st) {
    return by_widths(a, [&](auto n, auto p, auto full) {
        return backward<E, decltype(n)::value, decltype(p)::value, decltype(full)::value>(a, ws, st);
    });
}

}  // namespace
}  // namespace linattn
}  // namespace cssd
