// The gated delta rule over a sequence for 16-bit tensors, on the tcgen05
// tensor cores (the formulas stand at the head of delta.cu; the operand
// precision at the head of delta_tc.cuh).
//
// delta_prep_tc, one CTA per chunk and value head: [K; Q] K^T by one MMA
// chain, T = (I + A)^-1 and X = P T in fp32 on the CUDA cores, both left in
// the workspace as the very bytes the scan's B operand wants.
//
// delta_scan_tc, one CTA per value head, walks the chunks.  Everything is laid
// out transposed, one state column v per tensor-memory lane:
//     [v, i] = S^T K^T, S^T Q^T   A = S^T from tensor memory, B = K, Q
//     R^T = beta (V - e^G K S)^T  by the thread(s) of lane v
//     U^T, (X R)^T                A = R^T from tensor memory, B = T, X
//     S^T += U'^T K               A = U'^T from tensor memory, B = K^T
// so that each product's result lands in the lane whose thread makes the next
// A operand from it: rows never leave their lane, a row's scale needs no
// exchange beyond the two threads that share it, and no operand made on the
// way goes through shared memory.  Shared memory holds the B operands alone,
// two chunks deep, written by four loader warps (8 x 8 blocks: rows for K and
// Q, transposed in registers for K^T) and, for [T; X], by one bulk copy.
//
// What bounds the scan: the chain of a chunk, three MMA groups with the
// threads' work between them (the state is the only thing that waits; Q S and
// X R run beside the chain).

#include <atomic>

#include "delta_tc.cuh"

namespace cssd {
namespace delta {
namespace {

struct Shape {
    int T, H, G, N, P, nc;  // G: value heads per key head
};

// --------------------------------------------------------------- operands
// [K; Q]: rows i (64 of K, 64 of Q) by ND.  Column groups one 16-byte row
// apart from a multiple of 128, so that the lanes of a row group's column
// blocks store to different banks.
template <int ND>
struct KQ {
    static constexpr uint32_t SBO = 128, LBO = 16 * 128 + 16, BYTES = (ND / 8) * LBO;
    static constexpr uint32_t QROWS = 8 * SBO;  // bytes from K's rows to Q's
};
// K^T: rows k (ND) by 64 tokens, for the same reason with padded row groups.
template <int ND>
struct KT {
    static constexpr uint32_t SBO = 144, LBO = (ND / 8) * SBO, BYTES = 8 * LBO;
};

// One 8 x 8 block (8 tokens from `tok`, 8 columns): raw rows, zero where no
// token or column is.
template <typename E>
__device__ __forceinline__ void load_block(uint4 (&raw)[8], const E* src, int64_t stride, int tok, int n, bool cols) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
        raw[r] = (cols && tok + r < n) ? *reinterpret_cast<const uint4*>(src + (tok + r) * stride) : make_uint4(0, 0, 0, 0);
}
// The block scaled row by row (the scale is the row's over the CB lanes that
// hold its blocks) and packed to half; `down` gets the inverse scales.
template <typename E, int CB>
__device__ __forceinline__ void scale_block(const uint4 (&raw)[8], uint32_t (&w)[8][4], float (&down)[8]) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        uint32_t m = absmax2(absmax2(raw[r].x, raw[r].y), absmax2(raw[r].z, raw[r].w));
#pragma unroll
        for (int o = 1; o < CB; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        const RowScale s = row_scale(top_of<E>(m));
        down[r] = s.down;
        const uint32_t in[4] = {raw[r].x, raw[r].y, raw[r].z, raw[r].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 f = unpack2(in[c], E());
            w[r][c] = pack2(f.x * s.up, f.y * s.up);
        }
    }
}
// Rows as they are: row group rg, column block cb.
__device__ __forceinline__ void store_rows(unsigned char* base, uint32_t lbo, uint32_t sbo, int rg, int cb,
                                           const uint32_t (&w)[8][4]) {
    unsigned char* p = base + cb * lbo + rg * sbo;
#pragma unroll
    for (int r = 0; r < 8; ++r) *reinterpret_cast<uint4*>(p + 16 * r) = make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]);
}
// Transposed: columns become rows, the block's 8 tokens one 16-byte row.
__device__ __forceinline__ void store_transposed(unsigned char* base, uint32_t lbo, uint32_t sbo, int rg, int cb,
                                                 const uint32_t (&w)[8][4]) {
    unsigned char* p = base + rg * lbo + cb * sbo;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t sel = c & 1 ? 0x7632u : 0x5410u;
        *reinterpret_cast<uint4*>(p + 16 * c) =
            make_uint4(__byte_perm(w[0][c / 2], w[1][c / 2], sel), __byte_perm(w[2][c / 2], w[3][c / 2], sel),
                       __byte_perm(w[4][c / 2], w[5][c / 2], sel), __byte_perm(w[6][c / 2], w[7][c / 2], sel));
    }
}

// --------------------------------------------------------------- prep
constexpr int PT = 256;      // threads
constexpr int LT = C + 4;    // row stride of the fp32 matrices

template <int ND>
struct PrepSmem {
    static constexpr uint32_t STAGE = KQ<ND>::BYTES > Image::STRIDE ? KQ<ND>::BYTES : Image::STRIDE;
    static constexpr uint32_t A = STAGE, P = A + 4 * C * LT, T = P + 4 * C * LT, W = T + 4 * C * LT;
    static constexpr uint32_t BYTES = W + 4 * 32 * 32;
};

template <typename E, int ND>
__global__ void __launch_bounds__(PT) delta_prep_tc(const E* __restrict__ q, const E* __restrict__ k,
                                                    const float* __restrict__ g, const float* __restrict__ beta,
                                                    const int* __restrict__ lens, unsigned char* __restrict__ image,
                                                    Shape sh, unsigned* status) {
    using M = PrepSmem<ND>;
    constexpr int CB = ND / 8;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ Decays d;
    __shared__ float s_down[2 * C];
    __shared__ __align__(8) uint64_t mb[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x % sh.nc, bh = blockIdx.x / sh.nc;
    const int b = bh / sh.H, h = bh % sh.H, KH = sh.H / sh.G;
    const int n = min(row_len(lens, b, sh.T) - c * C, C);
    if (n <= 0) return;
    const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C;
    const int64_t ko = (t0 * KH + h / sh.G) * sh.N, ks = (int64_t)KH * sh.N;
    uint4 raw[8];
    const int which = tid / (8 * CB), rg = tid / CB % 8, cb = tid % CB;
    if (tid < 16 * CB) load_block(raw, (which ? q : k) + ko + 8 * cb, ks, 8 * rg, n, 8 * cb < sh.N);
    if (warp == 7) {
        tc::tmem_alloc(&s_tmem, 64);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        tc::mbar_init(&mb[0], 1);
        tc::mbar_init(&mb[1], 1);
        tc::mbar_fence_init();
        s_gave_up = 0;
    }
    if (tid < 16 * CB) {
        uint32_t w[8][4];
        float down[8];
        scale_block<E, CB>(raw, w, down);
        store_rows(smem, KQ<ND>::LBO, KQ<ND>::SBO, 8 * which + rg, cb, w);
        if (cb == 0)
#pragma unroll
            for (int r = 0; r < 8; ++r) s_down[C * which + 8 * rg + r] = down[r];
    }
    if (warp == 6) chunk_decays(d, g + t0 * sh.H + h, beta + t0 * sh.H + h, sh.H, n, lane);
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    if (tid == 0) {
        const uint64_t desc = tc::make_desc(tc::smem_u32(smem), KQ<ND>::LBO, KQ<ND>::SBO);
#pragma unroll
        for (int kk = 0; kk < ND / 16; ++kk) {
            const uint64_t at = desc + (uint64_t)((2 * kk * KQ<ND>::LBO) >> 4);
            tc::mma_f16(tmem, at, at, tc::idesc_f16(128, C), kk != 0);
        }
        tc::commit(&mb[0]);
    }
    float* sa = reinterpret_cast<float*>(smem + M::A);
    float* sp = reinterpret_cast<float*>(smem + M::P);
    float* st = reinterpret_cast<float*>(smem + M::T);
    float* sw = reinterpret_cast<float*>(smem + M::W);
    warp_wait(&mb[0], 0, &s_gave_up);
    tc::fence_after_sync();
    {  // lane i of tensor memory: row i of K (the first 64), of Q; columns j in halves
        const int row = 32 * (warp % 4) + lane, i = row % C, j0 = 32 * (warp / 4);
        uint32_t v[32];
        tmem_ld32(tmem + ((uint32_t)(32 * (warp % 4)) << 16) + j0, v);
        tc::tmem_wait_ld();
        const bool is_a = row < C;
        float* dst = (is_a ? sa : sp) + i * LT + j0;
        const float f = s_down[row] * (is_a ? d.beta[i] : 1.f);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int col = j0 + j + u;
                const bool keep = is_a ? i > col : i >= col;
                x[u] = keep ? __uint_as_float(v[j + u]) * s_down[col] * f * decay_between(d, i, col) : 0.f;
            }
            *reinterpret_cast<float4*>(dst + j) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
    __syncthreads();
    tri_inverse<LT>(sa, st, sw, tid);
    // X = P T, 4 x 4 a thread; then T's and X's rows as half pairs into the image
    const int ti = tid / 16, tj = tid % 16;
    float x[4][4] = {};
#pragma unroll 4
    for (int m = 0; m < C; m += 4) {
        float4 bv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) bv[u] = *reinterpret_cast<const float4*>(st + (m + u) * LT + 4 * tj);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float4 av = *reinterpret_cast<const float4*>(sp + (ti + 16 * r) * LT + m);
            const float a[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[r][0] = fmaf(a[u], bv[u].x, x[r][0]);
                x[r][1] = fmaf(a[u], bv[u].y, x[r][1]);
                x[r][2] = fmaf(a[u], bv[u].z, x[r][2]);
                x[r][3] = fmaf(a[u], bv[u].w, x[r][3]);
            }
        }
    }
    float* ff = reinterpret_cast<float*>(smem + Image::F);
    auto put = [&](int row, float (&e)[4]) {  // columns 4 tj.. of one row, held by the 16 threads of ti
        float top = fmaxf(fmaxf(fabsf(e[0]), fabsf(e[1])), fmaxf(fabsf(e[2]), fabsf(e[3])));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const RowScale s = row_scale(top);
        uint2 hi, lo;
        split2(e[0] * s.up, e[1] * s.up, hi.x, lo.x);
        split2(e[2] * s.up, e[3] * s.up, hi.y, lo.y);
        unsigned char* at = smem + (tj / 2) * Image::LBO + (row / 8) * Image::SBO + (row % 8) * 16 + (tj % 2) * 8;
        *reinterpret_cast<uint2*>(at) = hi;
        *reinterpret_cast<uint2*>(at + Image::PART) = lo;
        if (tj == 0) ff[Image::DOWN + row] = s.down;
    };
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float4 tv = *reinterpret_cast<const float4*>(st + (ti + 16 * r) * LT + 4 * tj);
        float e[4] = {tv.x, tv.y, tv.z, tv.w};
        put(ti + 16 * r, e);
        put(C + ti + 16 * r, x[r]);
    }
    if (tid < C) {
        ff[Image::IN + tid] = d.in[tid];
        ff[Image::OUT + tid] = d.out[tid];
        ff[Image::BETA + tid] = d.beta[tid];
    }
    if (tid < Image::FLOATS - Image::ALL) ff[Image::ALL + tid] = tid == 0 ? d.all : 0.f;
    __syncthreads();
    uint4* out = reinterpret_cast<uint4*>(image + (int64_t)blockIdx.x * Image::STRIDE);
    for (int e = tid; e < (int)(Image::BYTES / 16); e += PT) out[e] = reinterpret_cast<const uint4*>(smem)[e];
    if (tid == 0 && s_gave_up) {
        tc::drain_mmas(&mb[1], kDeltaWait);
        if (status) atomicOr(status, kStatusDelta);
    }
    __syncthreads();
    if (warp == 7) tc::tmem_dealloc(tmem, 64);
}

// --------------------------------------------------------------- scan
constexpr int CW = 8;                     // compute warps: two per lane quarter
constexpr int LW = 4;                     // loader warps
constexpr int ST = 32 * (CW + 1 + LW);    // threads (warp CW issues the MMAs)

template <int ND>
struct ScanSmem {
    static constexpr uint32_t KQ0 = 0, KT0 = KQ<ND>::BYTES, IMG = KT0 + KT<ND>::BYTES, V0 = IMG + Image::STRIDE;
    static constexpr uint32_t COEF = V0 + C * 128 * 2;
    // per-token factors: what v and the state's answer get in R, U and U'
    // from their products, and o's two parts
    static constexpr int VB = 0, KB = 64, UU = 128, UW = 192, OQ = 256, OX = 320, ALL = 384, DOWN = 388, FLOATS = 516;
    static constexpr uint32_t STAGE = (COEF + 4 * FLOATS + 15) / 16 * 16;
    static constexpr uint32_t BYTES = 2 * STAGE;
};

// Tensor-memory columns: the A operands, then the accumulators.  The state's
// update lies over K S and U, which are read before it is issued.
constexpr uint32_t COL_S = 0, COL_R = 128, COL_W = 192, COL_KS = 256, COL_U = 320, COL_D = 256, COL_QS = 384,
                   COL_X = 448, TMEM_COLS = 512;

// What the two warps of a lane quarter share: the larger of the two threads'
// largest values of a row, through shared memory, two slots in turn.
struct Pair {
    float (*slots)[2 * 128];
    uint64_t* bar;  // two arrivals a phase, one a warp
    int* gave_up;
    int half, v, n = 0;
    __device__ __forceinline__ float larger(float mine) {
        float* at = slots[n & 1];
        at[half * 128 + v] = mine;
        __syncwarp();
        if (v % 32 == 0) mbar_arrive(bar);
        warp_wait(bar, n & 1, gave_up);  // (a wait that gives up leaves a wrong scale; the chunk's next wait gives up too)
        ++n;
        return fmaxf(mine, at[(half ^ 1) * 128 + v]);
    }
};

// NE values of a lane's row (its other part is with the thread of the other
// half) scaled, split and stored as A-operand columns at `taddr` (hi) and
// `taddr + part` (lo); returns the inverse scale.
template <int NE>
__device__ __forceinline__ float store_operand(const float (&x)[NE], uint32_t taddr, uint32_t part, Pair& pair) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NE; i += 2) top = fmaxf(top, fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
    const RowScale s = row_scale(pair.larger(top));
#pragma unroll
    for (int c = 0; c < NE; c += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) split2(x[c + 2 * i] * s.up, x[c + 2 * i + 1] * s.up, hi[i], lo[i]);
        tc::tmem_st16(taddr + c / 2, hi);
        tc::tmem_st16(taddr + part + c / 2, lo);
    }
    tc::tmem_wait_st();
    return s.down;
}

// KEEP = false: outputs.  KEEP = true: the state entering each chunk and the
// writes U for the gradients, no outputs.
template <typename E, int ND, bool KEEP>
__global__ void __launch_bounds__(ST, 1) delta_scan_tc(const E* __restrict__ q, const E* __restrict__ k,
                                                       const E* __restrict__ v, const unsigned char* __restrict__ image,
                                                       const float* h0, const int* __restrict__ lens, float scale,
                                                       E* __restrict__ o, float* h_final, float* __restrict__ states,
                                                       float* __restrict__ writes, Shape sh, unsigned* status) {
    using M = ScanSmem<ND>;
    constexpr int CB = ND / 8, NS = ND / 2;  // NS: state elements a compute thread holds
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) uint64_t mb_full[2], mb_img[2], mb_free[2], mb_ks, mb_r, mb_u, mb_w, mb_d, mb_s, mb_pair[4],
        mb_load, mb_drain;
    __shared__ float s_top[2][2 * 128];
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bh = blockIdx.x, b = bh / sh.H, h = bh % sh.H, KH = sh.H / sh.G, N = sh.N, P = sh.P;
    const int len = row_len(lens, b, sh.T), nck = (len + C - 1) / C;
    const int live_warps = 2 * ((P + 31) / 32);
    if (warp == CW) {
        tc::tmem_alloc(&s_tmem, TMEM_COLS);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        s_gave_up = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&mb_full[i], LW);
            tc::mbar_init(&mb_img[i], 1);
            tc::mbar_init(&mb_free[i], live_warps);
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(&mb_pair[i], 2);
        tc::mbar_init(&mb_load, LW);
        tc::mbar_init(&mb_ks, 1);
        tc::mbar_init(&mb_u, 1);
        tc::mbar_init(&mb_d, 1);
        tc::mbar_init(&mb_drain, 1);
        tc::mbar_init(&mb_r, live_warps);
        tc::mbar_init(&mb_w, live_warps);
        tc::mbar_init(&mb_s, live_warps);
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;

    if (warp < CW) {
        // ------------------------------------------------ compute warps
        const int quarter = warp % 4, half = warp / 4, vc = 32 * quarter + lane;
        const bool on = vc < P;
        const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16);
        if (32 * quarter < P) {
            const int64_t so = (int64_t)bh * N * P + vc;
            const int k0 = half * NS;
            float s[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i) s[i] = (h0 && on && k0 + i < N) ? h0[so + (int64_t)(k0 + i) * P] : 0.f;
            Pair pair{s_top, &mb_pair[quarter], &s_gave_up, half, vc};
            float sdown = 1.f;
            auto done_with = [&](uint64_t* m) {  // this warp's tensor-memory accesses before the barrier are complete
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(m);
            };
            auto put_state = [&](int c) {
                if (KEEP && on) {
                    float* dst = states + ((int64_t)bh * sh.nc + c) * N * P + vc;
#pragma unroll
                    for (int i = 0; i < NS; ++i)
                        if (k0 + i < N) dst[(int64_t)(k0 + i) * P] = s[i];
                }
                sdown = store_operand<NS>(s, tq + COL_S + k0 / 2, ND / 2, pair);
                done_with(&mb_s);
            };
            if (nck > 0) put_state(0);
            for (int c = 0; c < nck; ++c) {
                const uint32_t ph = c & 1;
                unsigned char* stage = smem + (c & 1) * M::STAGE;
                const float* coef = reinterpret_cast<const float*>(stage + M::COEF) + 32 * half;
                if (!warp_wait(&mb_full[c & 1], (c >> 1) & 1, &s_gave_up)) break;
                const float all = reinterpret_cast<const float*>(stage + M::COEF)[M::ALL];
                const E* vt = reinterpret_cast<const E*>(stage + M::V0) + 32 * half * P + (on ? vc : 0);
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = to_f(vt[i * P]) * coef[M::VB + i];
                if (!warp_wait(&mb_ks, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                uint32_t raw[32];
                tmem_ld32(tq + COL_KS + 32 * half, raw);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = fmaf(-coef[M::KB + i] * sdown, __uint_as_float(raw[i]), x[i]);
                const float rdown = store_operand<32>(x, tq + COL_R + 16 * half, 32, pair);
                done_with(&mb_r);
                if (!warp_wait(&mb_u, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                tmem_ld32(tq + COL_U + 32 * half, raw);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(raw[i]) * rdown * coef[M::UW + i];
                const float wdown = store_operand<32>(x, tq + COL_W + 16 * half, 32, pair);
                done_with(&mb_w);
                if (KEEP && on) {
                    float* dst = writes + (((int64_t)bh * sh.nc + c) * C + 32 * half) * P + vc;
#pragma unroll
                    for (int i = 0; i < 32; ++i) dst[(int64_t)i * P] = __uint_as_float(raw[i]) * rdown * coef[M::UU + i];
                }
                if (!warp_wait(&mb_d, ph, &s_gave_up)) break;
                tc::fence_after_sync();
#pragma unroll
                for (int e = 0; e < NS; e += 32) {
                    tmem_ld32(tq + COL_D + k0 + e, raw);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[e + i] = fmaf(all, s[e + i], __uint_as_float(raw[i]) * wdown);
                }
                const float qdown = sdown;
                if (c + 1 < nck) put_state(c + 1);
                if constexpr (!KEEP) {
                    tmem_ld32(tq + COL_QS + 32 * half, raw);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(raw[i]) * (qdown * coef[M::OQ + i]);
                    tmem_ld32(tq + COL_X + 32 * half, raw);
                    tc::tmem_wait_ld();
                    const int n = min(len - c * C, C) - 32 * half;
                    E* dst = o + (((int64_t)b * sh.T + (int64_t)c * C + 32 * half) * sh.H + h) * P + vc;
                    const int64_t os = (int64_t)sh.H * P;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (on && i < n) dst[i * os] = from_f<E>(fmaf(__uint_as_float(raw[i]), rdown * coef[M::OX + i], x[i]));
                }
                done_with(&mb_free[c & 1]);
            }
            if (h_final && on)
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    if (k0 + i < N) h_final[so + (int64_t)(k0 + i) * P] = s[i];
            if (!KEEP && on)
                for (int t = len + half; t < sh.T; t += 2) o[(((int64_t)b * sh.T + t) * sh.H + h) * P + vc] = from_f<E>(0.f);
        }
    } else if (warp == CW) {
        // ------------------------------------------------ MMA issue
        if (lane == 0) {
            constexpr uint32_t id64 = tc::idesc_f16(128, C), idn = tc::idesc_f16(128, ND);
            for (int c = 0; c < nck; ++c) {
                const uint32_t ph = c & 1;
                const uint32_t base = tc::smem_u32(smem) + (c & 1) * M::STAGE;
                const uint64_t dkq = tc::make_desc(base + M::KQ0, KQ<ND>::LBO, KQ<ND>::SBO);
                const uint64_t dkt = tc::make_desc(base + M::KT0, KT<ND>::LBO, KT<ND>::SBO);
                const uint64_t dtx = tc::make_desc(base + M::IMG, Image::LBO, Image::SBO);
                auto chain = [&](uint32_t d, uint32_t a, uint64_t bd, uint32_t step, int kk, uint32_t id, bool first) {
                    for (int i = 0; i < kk; ++i) mma_f16_ts(d, a + 8 * i, bd + (uint64_t)((i * step) >> 4), id, !(first && i == 0));
                };
                if (!wait_or_give_up(&mb_full[c & 1], (c >> 1) & 1, &s_gave_up)) break;
                if (!wait_or_give_up(&mb_img[c & 1], (c >> 1) & 1, &s_gave_up)) break;
                if (!wait_or_give_up(&mb_s, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                for (int p = 0; p < 2; ++p)
                    chain(tmem + COL_KS, tmem + COL_S + p * (ND / 2), dkq, 2 * KQ<ND>::LBO, ND / 16, id64, p == 0);
                tc::commit(&mb_ks);
                if (!KEEP) {
                    if (c > 0 && !wait_or_give_up(&mb_free[(c - 1) & 1], ((c - 1) >> 1) & 1, &s_gave_up)) break;
                    tc::fence_after_sync();
                    for (int p = 0; p < 2; ++p)
                        chain(tmem + COL_QS, tmem + COL_S + p * (ND / 2), dkq + (KQ<ND>::QROWS >> 4), 2 * KQ<ND>::LBO, ND / 16,
                              id64, p == 0);
                }
                if (!wait_or_give_up(&mb_r, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                auto from_r = [&](uint32_t d, uint64_t bd) {  // hi hi + lo hi + hi lo
                    chain(d, tmem + COL_R, bd, 2 * Image::LBO, 4, id64, true);
                    chain(d, tmem + COL_R + 32, bd, 2 * Image::LBO, 4, id64, false);
                    chain(d, tmem + COL_R, bd + (Image::PART >> 4), 2 * Image::LBO, 4, id64, false);
                };
                from_r(tmem + COL_U, dtx);
                tc::commit(&mb_u);
                if (!KEEP) from_r(tmem + COL_X, dtx + ((8 * Image::SBO) >> 4));
                if (!wait_or_give_up(&mb_w, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                chain(tmem + COL_D, tmem + COL_W, dkt, 2 * KT<ND>::LBO, 4, idn, true);
                chain(tmem + COL_D, tmem + COL_W + 32, dkt, 2 * KT<ND>::LBO, 4, idn, false);
                tc::commit(&mb_d);
            }
            if (s_gave_up) tc::drain_mmas(&mb_drain, kDeltaWait);
        }
    } else {
        // ------------------------------------------------ loaders
        const int t = tid - 32 * (CW + 1);
        constexpr int NB = 2 * 8 * CB / 128;  // 8 x 8 blocks a thread
        int last[2] = {-1, -1};               // parity of the last copy into each stage
        for (int c = 0; c < nck; ++c) {
            unsigned char* stage = smem + (c & 1) * M::STAGE;
            float* coef = reinterpret_cast<float*>(stage + M::COEF);
            const int n = min(len - c * C, C);
            const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C;
            const int64_t ko = (t0 * KH + h / sh.G) * N, ks = (int64_t)KH * N;
            const unsigned char* img = image + ((int64_t)bh * sh.nc + c) * Image::STRIDE;
            const float* ff = reinterpret_cast<const float*>(img + Image::F);
            uint4 raw[NB][8], vr[8];
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const int id = t + 128 * e, which = id / (8 * CB), rg = id / CB % 8, cb = id % CB;
                load_block(raw[e], (which ? q : k) + ko + 8 * cb, ks, 8 * rg, n, 8 * cb < N && !(KEEP && which));
            }
            const int per = P / 8;  // 16-byte pieces of a row of V
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int id = t + 128 * e, i = id / per, p = id % per;
                vr[e] = (e < P / 16 && i < n) ? *reinterpret_cast<const uint4*>(v + ((t0 + i) * sh.H + h) * P + 8 * p)
                                              : make_uint4(0, 0, 0, 0);
            }
            float fi = 0.f, fo = 0.f, fb = 0.f, fu = 0.f, fx = 0.f;
            if (t < C) {
                fi = ff[Image::IN + t], fo = ff[Image::OUT + t], fb = ff[Image::BETA + t];
                fu = ff[Image::DOWN + t], fx = ff[Image::DOWN + C + t];
            }
            const float fa = ff[Image::ALL];
            if (c >= 2 && !warp_wait(&mb_free[c & 1], ((c >> 1) - 1) & 1, &s_gave_up)) break;
            if (t == 0) {
                tc::mbar_arrive_expect_tx(&mb_img[c & 1], Image::F);
                tc::bulk_g2s(tc::smem_u32(stage + M::IMG), img, Image::F, &mb_img[c & 1]);
                last[c & 1] = (c >> 1) & 1;
            }
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const int id = t + 128 * e, which = id / (8 * CB), rg = id / CB % 8, cb = id % CB;
                uint32_t w[8][4];
                float down[8];
                scale_block<E, CB>(raw[e], w, down);
                store_rows(stage + M::KQ0, KQ<ND>::LBO, KQ<ND>::SBO, 8 * which + rg, cb, w);
                if (which == 0) store_transposed(stage + M::KT0, KT<ND>::LBO, KT<ND>::SBO, rg, cb, w);
                if (cb == 0)
#pragma unroll
                    for (int r = 0; r < 8; ++r) coef[M::DOWN + C * which + 8 * rg + r] = down[r];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < P / 16) reinterpret_cast<uint4*>(stage + M::V0)[t + 128 * e] = vr[e];
            __syncwarp();
            if (lane == 0) mbar_arrive(&mb_load);
            if (!warp_wait(&mb_load, c & 1, &s_gave_up)) break;  // the row scales of all four warps
            if (t < C) {
                const float kd = coef[M::DOWN + t], qd = coef[M::DOWN + C + t];
                coef[M::VB + t] = fb;
                coef[M::KB + t] = fb * fi * kd;
                coef[M::UU + t] = fu;
                coef[M::UW + t] = fu * fo * kd;
                coef[M::OQ + t] = scale * fi * qd;
                coef[M::OX + t] = scale * fx;
                if (t == 0) coef[M::ALL] = fa;
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&mb_full[c & 1]);
        }
        if (t == 0 && s_gave_up)  // no copy may land in shared memory that is no longer this CTA's
            for (int i = 0; i < 2; ++i)
                if (last[i] >= 0) tc::mbar_wait_bounded(&mb_img[i], last[i], kDeltaWait);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == CW) tc::tmem_dealloc(tmem, TMEM_COLS);
    if (tid == 0 && s_gave_up && status) atomicOr(status, kStatusDelta);
}

Shape shape(const DeltaArgs& a) {
    return Shape{(int)a.T, (int)a.H, (int)(a.H / a.KH), (int)a.N, (int)a.P, (int)((a.T + C - 1) / C)};
}
int64_t chunk_count(const DeltaArgs& a) { return a.Bz * a.H * ((a.T + C - 1) / C); }

// Dynamic shared memory of kernel F, allowed once per device.
template <auto* F>
cudaError_t allow(uint32_t bytes) {
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

template <typename E, int ND>
cudaError_t forward_tc(const DeltaArgs& a, void* ws, cudaStream_t st) {
    unsigned char* image = static_cast<unsigned char*>(ws);
    unsigned* status = status_word();
    cudaError_t e = allow<delta_prep_tc<E, ND>>(PrepSmem<ND>::BYTES);
    if (e != cudaSuccess) return e;
    delta_prep_tc<E, ND><<<(unsigned)chunk_count(a), PT, PrepSmem<ND>::BYTES, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), a.g, a.beta, a.lens, image, shape(a), status);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = allow<delta_scan_tc<E, ND, false>>(ScanSmem<ND>::BYTES)) != cudaSuccess) return e;
    delta_scan_tc<E, ND, false><<<(unsigned)(a.Bz * a.H), ST, ScanSmem<ND>::BYTES, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.v), image, a.h0, a.lens, a.scale,
        static_cast<E*>(a.o), a.h_final, nullptr, nullptr, shape(a), status);
    return cudaGetLastError();
}

template <typename E>
cudaError_t forward_by_width(const DeltaArgs& a, void* ws, cudaStream_t st) {
    return a.N <= 64 ? forward_tc<E, 64>(a, ws, st) : forward_tc<E, 128>(a, ws, st);
}

}  // namespace

size_t tc_workspace_bytes(const DeltaArgs& a) { return (size_t)chunk_count(a) * Image::STRIDE; }
cudaError_t launch_forward_tc(const DeltaArgs& a, void* ws, cudaStream_t st) {
    return a.dtype == CSSD_BF16 ? forward_by_width<__nv_bfloat16>(a, ws, st) : forward_by_width<__half>(a, ws, st);
}

}  // namespace delta
}  // namespace cssd
