// Helpers of the linear-attention chunk kernels: values as bfloat16 planes, the
// warp-level matrix products over tiles in shared memory, and the decays of one
// chunk.
#pragma once

#include "delta_common.cuh"

namespace cssd {
namespace linattn {

using delta::add;
using delta::exp_of;
using delta::from_f;
using delta::row_len;
using delta::Sum2;
using delta::to_f;

// --------------------------------------------------------------- planes
// A value is held as a sum of bfloat16 planes, each the rounding of what the
// planes before it left: a bfloat16 is one plane, a half (11 significant bits)
// exactly two, a float (24 bits) exactly three.  bfloat16 has the exponents of
// float, so no plane needs a scale.  What the kernels make on the way (decayed
// keys, scores, states) is split the same way, and a product of two values takes
// the plane pairs (i, j) with i + j below a number of planes.
template <typename E>
struct Type;
template <>
struct Type<__nv_bfloat16> {
    static constexpr int NP = 1;
};
template <>
struct Type<__half> {
    static constexpr int NP = 2;
};
template <>
struct Type<float> {
    static constexpr int NP = 3;
};

__device__ __forceinline__ uint32_t pack_bf(float x, float y) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// x and y as NPL planes, two values a word.
template <int NPL>
__device__ __forceinline__ void split(float x, float y, uint32_t (&p)[NPL]) {
    p[0] = pack_bf(x, y);
#pragma unroll
    for (int i = 1; i < NPL; ++i) {
        x -= lo_f(p[i - 1]);
        y -= hi_f(p[i - 1]);
        p[i] = pack_bf(x, y);
    }
}

// --------------------------------------------------------------- tiles
// Rows of W columns, 2 bytes each, with 16 bytes between: eight rows then start
// in different banks, which is what ldmatrix wants.
constexpr int pitch(int w) { return 2 * w + 16; }

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
// A lane's address in a 16 x 16 block whose first element is (r0, c0): `FLIP` puts
// the second 8 rows into the third and fourth matrix (else into the second and
// fourth).
//   A [m][k]  ldsm    <false>      A stored [k][m]  ldsm_t  <true>
//   B [n][k]  ldsm    <true>       B stored [k][n]  ldsm_t  <false>
// (of B the registers 0, 1 are the first eight columns n, 2 and 3 the others)
template <bool FLIP>
__device__ __forceinline__ uint32_t lane_at(uint32_t base, int pitch_, int r0, int c0, int lane) {
    const int r = r0 + (lane & 7) + (FLIP ? (lane >> 4) * 8 : (lane >> 3 & 1) * 8);
    const int c = c0 + (FLIP ? (lane >> 3 & 1) * 8 : (lane >> 4) * 8);
    return base + r * pitch_ + 2 * c;
}
// The tiles of kernels with products on tcgen05 instead hold eight columns of all their rows after one another, 16 bytes a row: blocks
// of 8 x 8 are 128 contiguous bytes, which ldmatrix reads without conflicts and the tcgen05 descriptors take as they
// are, either way round.  16 bytes between the groups of columns let a row be written without conflicts too.  (The
// kernels without such products are slower on these tiles, whose rows a copy writes to eight places: 75 us against 65 for the
// forward of 4 x 2048 x 24, 64/64.)
__host__ __device__ constexpr int group_bytes(int rows) { return 16 * rows + 16; }
__host__ __device__ constexpr int plane_bytes(int rows, int w) { return w / 8 * group_bytes(rows); }
// As lane_at, for a tile of ROWS rows.
template <bool FLIP, int ROWS>
__device__ __forceinline__ uint32_t core_at(uint32_t base, int r0, int c0, int lane) {
    const int r = r0 + (lane & 7) + (FLIP ? (lane >> 4) * 8 : (lane >> 3 & 1) * 8);
    const int cg = c0 / 8 + (FLIP ? (lane >> 3 & 1) : (lane >> 4));
    return base + cg * group_bytes(ROWS) + 16 * r;
}
// Where a block of 16 tokens lies among a tile's rows.  TC (128 rows, products on tcgen05): the blocks b and 7 - b lie
// side by side, in the 32 lanes of tensor memory that the two warps which have them may read.
template <bool TC>
__device__ __forceinline__ int place(int block) {
    return TC ? (block < 4 ? 2 * block : 15 - 2 * block) : block;
}
// A tile of ROWS rows of W columns in either layout (TC: the core one): the bytes of a plane and from 16 columns to
// the next, and a lane's address in the 16 x 16 block of tokens `block`, columns c0..
template <bool TC, int ROWS, int W>
struct Tile {
    static constexpr int PLANE = TC ? plane_bytes(ROWS, W) : ROWS * pitch(W), STEP = TC ? 2 * group_bytes(ROWS) : 32;
    template <bool FLIP>
    static __device__ __forceinline__ uint32_t at(uint32_t base, int block, int c0, int lane) {
        if constexpr (TC)
            return core_at<FLIP, ROWS>(base, 16 * place<ROWS == 128>(block), c0, lane);
        else
            return lane_at<FLIP>(base, pitch(W), 16 * block, c0, lane);
    }
};
// c = A B (the sum's first 16), and c += A B, for 16 x 8 outputs.
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
    const int bytes = there ? 16 : 0;  // (nothing is read where it is not; the rest is zero)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ROWS tokens of `width` columns (a multiple of 16, at most W; rows from n on are zeros) into the planes at `dst`,
// `plane` bytes apart.  bfloat16 comes by cp.async (the caller commits and waits), the others through registers.
template <typename E, int W, int ROWS, int NT>
__device__ __forceinline__ void load_tile(unsigned char* dst, int plane, const E* src, int64_t stride, int n, int width, int tid) {
    constexpr int NP = Type<E>::NP, V = 16 / sizeof(E), PER = W / V, STEP = NT / PER;
    static_assert(NT % PER == 0 && ROWS % STEP == 0, "whole rows a step");
    const int r0 = tid / PER, c = tid % PER;
    if (c * V >= width) return;
    src += r0 * stride + c * V;
    const int64_t step = STEP * stride;
    if constexpr (NP == 1) {
        uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst)) + r0 * pitch(W) + 16 * c;
        n -= r0;
#pragma unroll
        for (int r = 0; r < ROWS; r += STEP, src += step) cp16(to + r * pitch(W), src, r < n);
    } else {
        unsigned char* at = dst + r0 * pitch(W) + c * V * 2;
#pragma unroll
        for (int r = 0; r < ROWS; r += STEP, at += STEP * pitch(W), src += step) {
            alignas(16) E e[V];
            *reinterpret_cast<uint4*>(e) = r0 + r < n ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
            uint32_t w[NP][V / 2];
#pragma unroll
            for (int u = 0; u < V / 2; ++u) {
                uint32_t p[NP];
                split<NP>(to_f(e[2 * u]), to_f(e[2 * u + 1]), p);
#pragma unroll
                for (int z = 0; z < NP; ++z) w[z][u] = p[z];
            }
#pragma unroll
            for (int z = 0; z < NP; ++z) {
                if constexpr (V == 8)
                    *reinterpret_cast<uint4*>(at + z * plane) = make_uint4(w[z][0], w[z][1], w[z][2], w[z][3]);
                else
                    *reinterpret_cast<uint2*>(at + z * plane) = make_uint2(w[z][0], w[z][1]);
            }
        }
    }
}

// 128 tokens of `width` bfloat16 columns (at most W; rows from n on are zeros) into a core tile, by NT threads.
template <int W, int NT>
__device__ __forceinline__ void load_core(unsigned char* dst, const __nv_bfloat16* src, int64_t stride, int n, int width, int tid) {
    constexpr int PER = W / 8, STEP = NT / PER;
    const int t0 = tid / PER, col = tid % PER * 8;
    if (col >= width) return;
    src += t0 * stride + col;
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst)) + col / 8 * group_bytes(128);
#pragma unroll
    for (int t = 0; t < 128; t += STEP, src += STEP * stride)
        cp16(to + 16 * (16 * place<true>((t0 + t) / 16) + (t0 + t) % 16), src, t0 + t < n);
}

// Division of n < 2^31 by a number that is the same all over a launch.
struct Divisor {
    uint32_t d, m, s;
    __host__ static Divisor of(uint32_t d) {
        uint32_t s = 0;
        while ((1ull << s) < d) ++s;
        return {d, (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s};
    }
    __device__ __forceinline__ int div(int n, int& rest) const {
        const uint32_t q = (__umulhi(m, (uint32_t)n) + (uint32_t)n) >> s;
        rest = (int)((uint32_t)n - q * d);
        return (int)q;
    }
};

// --------------------------------------------------------------- decays
// G_i is the running sum of the log decays of a chunk.  The decay between two
// tokens j < i of different blocks of 16 is taken as three factors,
//     exp(G_i - G_j) = e_i X[block of j][block of i] f_j
// (from the block's start through i; between the blocks; from j to its block's
// end), none of which can overflow where the product does not, for g <= 0; in a
// block it is exp of the difference.  Sums are kept as two floats: the
// differences have to be right to an absolute 1e-7 while the sums reach hundreds.
template <int C>
struct alignas(16) Decays {
    static constexpr int NB = C / 16;
    float hi[C], lo[C];  // G_i
    float in[C];         // exp(G_i)
    float e[C], f[C];
    float x[NB][NB];
    float all, unused[3];  // exp(G_end)
    float out[C];        // exp(G_end - G_i); (last: the outputs do without it)
};

// The running sums of a chunk's log decays, K = C / 32 consecutive tokens a lane.
template <int C>
struct Sums {
    static constexpr int K = C / 32;
    Sum2 G[K];
    Sum2 end;
};
// One warp.  Tokens at or past n count as g = 0.  g is of the chunk's first token, `stride` elements between tokens
// (0: one decay for all).  A log decay of -inf counts as -1000, whose exponential is 0 too, so that differences
// stay numbers.
template <int C>
__device__ __forceinline__ Sums<C> chunk_sums(const float* g, int64_t stride, int n, int lane) {
    constexpr int K = C / 32;
    Sums<C> s;
    float gv[K];
#pragma unroll
    for (int e = 0; e < K; ++e) gv[e] = K * lane + e < n ? g[(K * lane + e) * stride] : 0.f;
#pragma unroll
    for (int e = 0; e < K; ++e) {
        s.G[e] = {gv[e] < -1000.f ? -1000.f : gv[e], 0.f};
        if (e) s.G[e] = add(s.G[e - 1], s.G[e]);
    }
    Sum2 tot = s.G[K - 1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum2 up = {__shfl_up_sync(0xffffffffu, tot.hi, o), __shfl_up_sync(0xffffffffu, tot.lo, o)};
        if (lane >= o) tot = add(up, tot);
    }
    Sum2 before = {__shfl_up_sync(0xffffffffu, tot.hi, 1), __shfl_up_sync(0xffffffffu, tot.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    s.end = {__shfl_sync(0xffffffffu, tot.hi, 31), __shfl_sync(0xffffffffu, tot.lo, 31)};
#pragma unroll
    for (int e = 0; e < K; ++e) s.G[e] = add(before, s.G[e]);
    return s;
}
// exp(s) as two floats.  A state is multiplied by the decays of as many chunks (of one token's, step by step) as it
// remembers, and with one decay a head all of them are off the same way: by up to 2^-23 of itself each time for a float
// (at g = -3e-4 the states of 5000 tokens were off by 2e-6 in the 2-norm, after 4000 single tokens by 4e-5; with both
// floats by less than 1e-6 and 2e-6, times unchanged within 0.5 %).  Near 1, where states remember, the second float is
// what expm1, right to its own 2^-23, has beside the first one's distance from 1.
__device__ __forceinline__ float2 exp_pair(Sum2 s) {
    const float e = exp_of(s);
    if (!(fabsf(s.hi) < 0.6f)) return make_float2(e, 0.f);
    const float m = expm1f(s.hi);
    return make_float2(e, fmaf(1.f + m, s.lo, m) - (e - 1.f));  // (e - 1 is exact)
}
__device__ __forceinline__ float exp_between(Sum2 a, Sum2 b) { return exp_of(add(a, {-b.hi, -b.lo})); }

// The chunk's tables from its sums, by one warp, into memory of any kind.
template <int C>
__device__ __forceinline__ void put_decays(Decays<C>& d, const Sums<C>& s, int lane) {
    constexpr int K = C / 32, LPB = 16 / K, NB = C / 16;  // lanes per block of 16 tokens
    const Sum2 tot = s.G[K - 1];
    auto of_lane = [&](int l) {  // the sum through lane l's last token (l -1: none)
        const Sum2 v = {__shfl_sync(0xffffffffu, tot.hi, l < 0 ? 0 : l), __shfl_sync(0xffffffffu, tot.lo, l < 0 ? 0 : l)};
        return l < 0 ? Sum2{0.f, 0.f} : v;
    };
    const Sum2 first = of_lane(lane / LPB * LPB - 1), last = of_lane(lane / LPB * LPB + LPB - 1);
#pragma unroll
    for (int e = 0; e < K; ++e) {
        const int i = K * lane + e;
        d.hi[i] = s.G[e].hi;
        d.lo[i] = s.G[e].lo;
        d.in[i] = exp_of(s.G[e]);
        d.out[i] = exp_between(s.end, s.G[e]);
        d.e[i] = exp_between(s.G[e], first);
        d.f[i] = exp_between(last, s.G[e]);
    }
#pragma unroll
    for (int i0 = 0; i0 < NB * NB; i0 += 32) {
        const int i = i0 + lane, a = i / NB % NB, b = i % NB;
        const Sum2 end = of_lane(a * LPB + LPB - 1), start = of_lane(b * LPB - 1);
        if (i < NB * NB) (&d.x[0][0])[i] = a < b ? exp_between(start, end) : 0.f;
    }
    if (lane == 0) d.all = exp_of(s.end);
}

}  // namespace linattn
}  // namespace cssd
