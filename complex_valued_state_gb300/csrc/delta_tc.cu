// The gated delta rule over a sequence for 16-bit tensors, on the tcgen05
// tensor cores (the formulas stand at the head of delta.cu; the operand
// precision at the head of delta_tc.cuh).
//
// delta_prep_tc, one CTA per chunk and value head: [Q; K] K^T by one MMA
// chain, T = (I + A)^-1 and X = P T in fp32 on the CUDA cores, all left in the
// workspace as the very bytes the scan's B operands want.
//
// delta_scan_tc, one CTA per value head, walks the chunks.  Everything is laid
// out transposed, one state column v per tensor-memory lane:
//     [v, i] = S^T K^T, S^T Q^T   A = S^T from tensor memory, B = K, Q
//     R^T = (V - e^G K S)^T       by the four threads of lane v
//     U^T, (X R)^T                A = R^T from tensor memory, B = T, X (times beta)
//     S^T += U'^T K               A = U'^T from tensor memory, B = K^T
// so that each product's result lands in the lane whose threads make the next
// A operand from it: rows never leave their lane, and no operand made on the
// way goes through shared memory.  Shared memory holds the B operands alone,
// two chunks deep, by bulk copies of what the prep left, and V or dO on a ring
// of its own.
//
// What bounds the scan: the chain of a chunk, three MMA groups with the
// threads' work between them (the state is the only thing that waits; Q S and
// X R run beside the chain).  A chunk takes 2.6 us at 64/64, 3.5 at 128/64 and 3.9
// at 128/128 (what a row of 4 heads takes more for each); the tensor pipe is 15 %
// busy.
//
// Whole calls, bf16: forward 4 x 2048 x 24, 64/64 189 us (prep 107 us alone, half
// of it beside the scan); 1 x 16384 x 32, 128/64 1058 us; gradients 4 x 2048 x 24,
// 64/64 535 us (prep 115, scans 209, delta_grad_tc 211), 4 x 1501 x 16 on 8 key
// heads, 128/128 356 us (45, 114, 176 and 21 for the sum over shared heads).

#include <type_traits>

#include "delta_tc.cuh"

namespace cssd {
namespace delta {
namespace {

struct Shape {
    int T, H, G, N, P, nc;  // G: value heads per key head
    int c0, c1;             // the chunks of this launch
};

// --------------------------------------------------------------- operands
// Half a row (ND / 2 columns) scaled and packed; the scale is the row's over
// the two lanes that hold it.  Stores into the operand's row `r`, returns the
// inverse scale.
template <typename E, int ND>
__device__ __forceinline__ float store_half_row(const uint4 (&raw)[ND / 16], unsigned char* base, int r, int part) {
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < ND / 16; ++g)
        m = __vmaxu2(m, __vmaxu2(absmax2(raw[g].x, raw[g].y), absmax2(raw[g].z, raw[g].w)));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const RowScale s = row_scale(top_of<E>(m));
    unsigned char* p = base + (r / 8) * QK<ND>::SBO + (r % 8) * 16 + part * (ND / 16) * QK<ND>::LBO;
#pragma unroll
    for (int g = 0; g < ND / 16; ++g) {
        const uint32_t in[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 f = unpack2(in[c], E());
            w[c] = pack2(f.x * s.up, f.y * s.up);
        }
        *reinterpret_cast<uint4*>(p + g * QK<ND>::LBO) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return s.down;
}
// The transposed operand (rows k, 64 tokens) of 64 rows of the operand at
// `from`, whose first row is `row0`: 8 x 8 blocks through ldmatrix, a warp four at a
// time, 128 contiguous bytes a block either way.
template <int ND>
__device__ __forceinline__ void transpose_operand(unsigned char* to, const unsigned char* from, int row0, int warp,
                                                  int warps, int lane) {
    for (int q = warp; q < 2 * (ND / 8); q += warps) {  // column block q / 2, token blocks 4 (q % 2)..
        const int cb = q / 2, tb = 4 * (q % 2);
        const uint32_t at = tc::smem_u32(from) + cb * QK<ND>::LBO + (row0 / 8 + tb + lane / 8) * QK<ND>::SBO + (lane % 8) * 16;
        uint32_t w[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(at)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint32_t*>(to + (tb + i) * KT<ND>::LBO + cb * KT<ND>::SBO + (lane / 4) * 16 + (lane % 4) * 4) = w[i];
    }
}

// --------------------------------------------------------------- prep
// Bound by instruction issue (59 % busy) and the barriers between its stages
// (the loads, the MMA, the inverse, X, the image): 35 ns a chunk and head at 64/64
// forward, 37 for the gradients, whose second image stands for the outputs' X.
constexpr int PT = 256;      // threads
constexpr int LT = C + 4;    // row stride of the fp32 matrices

template <int ND, bool BACK>
struct PrepSmem {
    // The operands of K and Q; once they are read, A (then T) and P (then X)
    // lie over them, and over those the images, when T and X are in registers.
    static constexpr uint32_t OPS = BACK ? Operands<ND>::BWD : Operands<ND>::FWD;
    static constexpr uint32_t A = 0, P = 4 * C * LT, W = 2 * P;
    static constexpr uint32_t mx(uint32_t a, uint32_t b) { return a > b ? a : b; }
    static constexpr uint32_t BYTES = mx(mx(OPS, W + 4 * kInverseScratch), Image::STRIDE);
};

// 16 values of a row of the image (columns 16 part..), scaled and split; returns
// the sum of their absolute values.
__device__ __forceinline__ float image_row(unsigned char* img, int row, int part, const float (&e)[16], float up) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float a = e[8 * g + 2 * u], b = e[8 * g + 2 * u + 1];
            sum += fabsf(a) + fabsf(b);
            split2(a * up, b * up, h[u], l[u]);
        }
        unsigned char* at = img + (2 * part + g) * Image::LBO + (row / 8) * Image::SBO + (row % 8) * 16;
        *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(at + Image::PART) = make_uint4(l[0], l[1], l[2], l[3]);
    }
    return sum;
}

// One warp: the chunk's decay and the larger of its lanes' bounds.
__device__ __forceinline__ void put_scalars(float* ff, float all, float b1, float b2, float b3, int lane) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, o));
        b2 = fmaxf(b2, __shfl_xor_sync(0xffffffffu, b2, o));
        b3 = fmaxf(b3, __shfl_xor_sync(0xffffffffu, b3, o));
    }
    if (lane == 0) {
        ff[Image::ALL] = all;
        ff[Image::BND1] = b1;
        ff[Image::BND2] = b2;
        ff[Image::BND3] = b3;
    }
}

// BACK: a second image for the backward scan, [T^T; X^T].
template <typename E, int ND, bool BACK>
__global__ void __launch_bounds__(PT, BACK ? 3 : 4) delta_prep_tc(const E* __restrict__ q, const E* __restrict__ k,
                                                       const float* __restrict__ g, const float* __restrict__ beta,
                                                       const int* __restrict__ lens, unsigned char* __restrict__ image,
                                                       unsigned char* __restrict__ image_t,
                                                       unsigned char* __restrict__ operands, float scale, Shape sh,
                                                       unsigned* status) {
    using M = PrepSmem<ND, BACK>;
    using O = Operands<ND>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(16) Decays d;
    __shared__ __align__(16) float s_down[2 * C];  // inverse scales of K's and Q's rows
    __shared__ float s_sum[4][C], s_sumx[4][C];   // parts of sums over T's and X's rows (columns)
    __shared__ float s_norm[C];                   // |k|
    __shared__ float s_top[4][PT / 32];
    __shared__ __align__(16) DecayTables tab;
    __shared__ __align__(8) uint64_t mb[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = sh.c0 + blockIdx.x % (sh.c1 - sh.c0), bh = blockIdx.x / (sh.c1 - sh.c0);
    const int b = bh / sh.H, h = bh % sh.H, KH = sh.H / sh.G;
    const int n = min(row_len(lens, b, sh.T) - c * C, C);
    // A launch that overlaps the scan before it (see forward_tc) ends no sooner
    // than that scan, so that what follows in the stream comes after both.
    const bool last_block = blockIdx.x == gridDim.x - 1;
    if (n <= 0) {
        if (last_block) wait_for_previous();
        return;
    }
    const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C, ci = (int64_t)bh * sh.nc + c;
    const int64_t ko = (t0 * KH + h / sh.G) * sh.N, ks = (int64_t)KH * sh.N;
    uint4 raw[ND / 16];  // half a row: of Q's token tid / 2, or of K's
    const int qrow = tid / 2, half = tid % 2, tok = qrow % C;
    {
        const E* src = (qrow < C ? q : k) + ko + tok * ks + half * (ND / 2);
#pragma unroll
        for (int g = 0; g < ND / 16; ++g)
            raw[g] = tok < n && half * (ND / 2) + 8 * g < sh.N ? *reinterpret_cast<const uint4*>(src + 8 * g) : make_uint4(0, 0, 0, 0);
    }
    if (warp == 7) {
        tc::tmem_alloc(&s_tmem, 64);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        tc::mbar_init(&mb[0], 1);
        tc::mbar_init(&mb[1], 1);
        tc::mbar_fence_init();
        s_gave_up = 0;
        tab.steep = 0;
    }
    {
        const float down = store_half_row<E, ND>(raw, smem, qrow, half);
        if (half == 0) s_down[qrow < C ? C + tok : tok] = down;  // (K's first)
    }
    if (warp == 6) chunk_decays(d, g + t0 * sh.H + h, beta + t0 * sh.H + h, sh.H, n, lane);
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    if (tid == 0) {
        const uint64_t desc = tc::make_desc(tc::smem_u32(smem), QK<ND>::LBO, QK<ND>::SBO);
#pragma unroll
        for (int kk = 0; kk < ND / 16; ++kk) {
            const uint64_t at = desc + (uint64_t)((2 * kk * QK<ND>::LBO) >> 4);
            tc::mma_f16(tmem, at, at + (QK<ND>::KROWS >> 4), tc::idesc_f16(128, C), kk != 0);
        }
        tc::commit(&mb[0]);
    }
    float* sa = reinterpret_cast<float*>(smem + M::A);  // A, then T in its place
    float* sp = reinterpret_cast<float*>(smem + M::P);
    decay_tables(tab, d, s_down, tid);  // while the MMA runs
    const bool owner = h % sh.G == 0;  // this CTA leaves the key head's operands, once for its group
    if (owner) {
        transpose_operand<ND>(smem + O::KT0, smem, C, warp, PT / 32, lane);
        if (BACK) transpose_operand<ND>(smem + O::QT0, smem, 0, warp, PT / 32, lane);
        tc::fence_proxy_async();
    }
    __syncthreads();
    if (tid == 0 && owner) {
        bulk_s2g(operands + (((int64_t)b * KH + h / sh.G) * sh.nc + c) * M::OPS, tc::smem_u32(smem), M::OPS);
        bulk_commit();
    }
    {  // lane i of tensor memory: row i of Q (the first 64), of K; columns j in halves
        const int row = 32 * (warp % 4) + lane, i = row % C, j0 = 32 * (warp / 4);
        const bool is_a = row >= C;
        float* dst = (is_a ? sa : sp) + i * LT + j0;
        const bool above = 32 * (warp % 2) < j0;  // every pair of this warp has i < j
        uint32_t v[32];
        warp_wait(&mb[0], 0, &s_gave_up);
        tc::fence_after_sync();
        tmem_ld32(tmem + ((uint32_t)(32 * (warp % 4)) << 16) + j0, v);
        tc::tmem_wait_ld();
        const float f = is_a ? s_down[i] * d.beta[i] : s_down[C + i];
        const int last = is_a ? i - 1 : i;  // the row's last column that is not zero
        float x[32];
        if (is_a && i / 32 == j0 / 32) {  // (K K^T)_ii: beside the diagonal's own scale
            float diag = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) diag = j0 + j == i ? __uint_as_float(v[j]) : diag;
            s_norm[i] = sqrtf(diag) * s_down[i];
        }
        if (above) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = 0.f;
        } else if (!tab.steep) {
            const float fe = f * tab.e[i];
            const float4* fj = reinterpret_cast<const float4*>(tab.f[i / 16] + j0);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 m = fj[j / 4];
                x[j] = j0 + j <= last ? __uint_as_float(v[j]) * (m.x * fe) : 0.f;
                x[j + 1] = j0 + j + 1 <= last ? __uint_as_float(v[j + 1]) * (m.y * fe) : 0.f;
                x[j + 2] = j0 + j + 2 <= last ? __uint_as_float(v[j + 2]) * (m.z * fe) : 0.f;
                x[j + 3] = j0 + j + 3 <= last ? __uint_as_float(v[j + 3]) * (m.w * fe) : 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[j] = j0 + j <= last ? __uint_as_float(v[j]) * (s_down[j0 + j] * f) * steep_decay(d, i, j0 + j) : 0.f;
        }
        if (tid == 0) bulk_wait_read();  // the operands are copied out: their memory is free
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(dst + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    }
    __syncthreads();
    tri_inverse_in_place<LT>(sa, reinterpret_cast<float*>(smem + M::W), tid);
    // X = P T (both lower triangular), 8 x 4 to two neighbouring lanes that share
    // the sum (1.5 bytes of shared memory a multiply-add; 4 x 4, 2): a warp holds
    // 8 rows and stops at their last column
    const int l = tid & 1, tj = tid / 2 % 16;
    float x[8][4] = {};
#pragma unroll 1
    for (int m = 4 * l; m < 8 * (warp + 1); m += 8) {
        float4 bv[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) bv[u] = *reinterpret_cast<const float4*>(sa + (m + u) * LT + 4 * tj);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float4 av = *reinterpret_cast<const float4*>(sp + (8 * warp + r) * LT + m);
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
    join<2>(x, l);
    unsigned char* img = smem;
    float* ff = reinterpret_cast<float*>(img + Image::F);
    auto write_out = [&](unsigned char* to) {
        tc::fence_proxy_async();
        __syncthreads();
        if (tid == 0) {
            bulk_s2g(to + ci * Image::STRIDE, tc::smem_u32(img), Image::BYTES);
            bulk_commit();
            bulk_wait_read();
        }
    };
    __syncthreads();  // P is read
#pragma unroll
    for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4*>(sp + (8 * warp + 4 * l + r) * LT + 4 * tj) = make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
    __syncthreads();
    // T and X into the image: a thread has 16 columns of one row.  One scale a
    // matrix: the scales have 2^16 to spare.
    const int row = lane + 32 * (warp & 1), part = warp >> 1;
    // (The gradients' forward scan makes no outputs: X's part of its image is copied
    // as it lies here and not read.)
    float te[16], xe[BACK ? 1 : 16], tops[4] = {};  // of beta T, beta X; of T, X
#pragma unroll
    for (int u = 0; u < 16; u += 4) {
        const float4 t4 = *reinterpret_cast<const float4*>(sa + row * LT + 16 * part + u);
        const float4 x4 = *reinterpret_cast<const float4*>(sp + row * LT + 16 * part + u);
        const float4 b4 = *reinterpret_cast<const float4*>(d.beta + 16 * part + u);
        te[u] = t4.x * b4.x, te[u + 1] = t4.y * b4.y, te[u + 2] = t4.z * b4.z, te[u + 3] = t4.w * b4.w;
        if constexpr (!BACK) {
            xe[u] = x4.x * b4.x, xe[u + 1] = x4.y * b4.y, xe[u + 2] = x4.z * b4.z, xe[u + 3] = x4.w * b4.w;
            tops[1] = fmaxf(fmaxf(fmaxf(tops[1], fabsf(xe[u])), fmaxf(fabsf(xe[u + 1]), fabsf(xe[u + 2]))), fabsf(xe[u + 3]));
        }
        tops[0] = fmaxf(fmaxf(fmaxf(tops[0], fabsf(te[u])), fmaxf(fabsf(te[u + 1]), fabsf(te[u + 2]))), fabsf(te[u + 3]));
        if (BACK) {
            tops[2] = fmaxf(fmaxf(fmaxf(tops[2], fabsf(t4.x)), fmaxf(fabsf(t4.y), fabsf(t4.z))), fabsf(t4.w));
            tops[3] = fmaxf(fmaxf(fmaxf(tops[3], fabsf(x4.x)), fmaxf(fabsf(x4.y), fabsf(x4.z))), fabsf(x4.w));
        }
    }
    float tt[BACK ? 16 : 1], xt[BACK ? 16 : 1];  // of the transposes, for the second image
    if constexpr (BACK)
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            tt[u] = sa[(16 * part + u) * LT + row];
            xt[u] = sp[(16 * part + u) * LT + row];
        }
    constexpr int NTOP = BACK ? 4 : 2;
#pragma unroll
    for (int e = 0; e < NTOP; ++e) {
        // (non-negative: the order of the bits; a NaN is the largest)
        tops[e] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(tops[e])));
        if (lane == 0) s_top[e][warp] = tops[e];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < NTOP; ++e)
#pragma unroll
        for (int w = 0; w < PT / 32; ++w) tops[e] = fmaxf(tops[e], s_top[e][w]);
    RowScale ts = row_scale(tops[0]), xs = row_scale(tops[1]);
    // (the forward's matrices carry beta: U = T beta (V - e^G K S))
    s_sum[part][row] = image_row(img, row, part, te, ts.up);
    if constexpr (!BACK) image_row(img, C + row, part, xe, xs.up);
    __syncthreads();
    // |R| <= |v| + BND1 |S| and |U'| <= BND2 |R|, of a lane's largest values
    auto bound2 = [&](int i, const float* f) {
        return ((s_sum[0][i] + s_sum[1][i]) + (s_sum[2][i] + s_sum[3][i])) * f[i] * s_down[i];
    };
    if (tid < C) {
        const float kd = s_down[tid], qd = s_down[C + tid], fi = d.in[tid];
        ff[Image::KB + tid] = fi * kd;
        ff[Image::UU + tid] = ts.down;
        ff[Image::UW + tid] = ts.down * d.out[tid] * kd;
        if (!BACK) {
            ff[Image::OQ + tid] = scale * fi * qd;
            ff[Image::OX + tid] = scale * xs.down;
        }
    } else if (warp == 2) {
        put_scalars(ff, d.all, fmaxf(s_norm[lane] * d.in[lane], s_norm[lane + 32] * d.in[lane + 32]) * sqrtf((float)sh.N),
                    fmaxf(bound2(lane, d.out), bound2(lane + 32, d.out)), 0.f, lane);
    }
    write_out(image);
    if constexpr (BACK) {
        __syncthreads();  // (the first is copied out)
        ts = row_scale(tops[2]), xs = row_scale(tops[3]);
        s_sum[part][row] = image_row(img, row, part, tt, ts.up);
        s_sumx[part][row] = image_row(img, C + row, part, xt, xs.up);
        __syncthreads();
        if (tid < C) {
            const float kd = s_down[tid], qd = s_down[C + tid], fi = d.in[tid];
            ff[Image::WK + tid] = d.out[tid] * kd;
            ff[Image::ZT + tid] = ts.down;
            ff[Image::ZX + tid] = scale * xs.down;
            ff[Image::RZ + tid] = -fi * d.beta[tid] * kd;
            ff[Image::DQ + tid] = scale * fi * qd;
            ff[Image::KD + tid] = kd;
            ff[Image::QD + tid] = qd;
        } else if (warp == 2) {
            // |W| <= BND1 |dS|, the second operand <= BND2 |W| + BND3 |dO|, of a lane's largest values
            float b1 = 0.f, b2 = 0.f, b3 = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = lane + 32 * e;
                const float f = d.in[i] * fabsf(d.beta[i]) * s_down[i];
                b1 = fmaxf(b1, s_norm[i] * d.out[i]);
                b2 = fmaxf(b2, f * ((s_sum[0][i] + s_sum[1][i]) + (s_sum[2][i] + s_sum[3][i])));
                b3 = fmaxf(b3, f * fabsf(scale) * ((s_sumx[0][i] + s_sumx[1][i]) + (s_sumx[2][i] + s_sumx[3][i])));
            }
            put_scalars(ff, d.all, b1 * sqrtf((float)sh.N), b2, b3, lane);
        }
        write_out(image_t);
    }
    if (tid == 0) bulk_wait();
    if (tid == 0 && s_gave_up) {
        tc::drain_mmas(&mb[1], kDeltaWait);
        if (status) atomicOr(status, kStatusDelta);
    }
    __syncthreads();
    if (warp == 7) tc::tmem_dealloc(tmem, 64);
    if (last_block) wait_for_previous();
}

// --------------------------------------------------------------- scan
constexpr int PARTS = 4;       // threads that share a lane's row on the chain
constexpr int CW = 4 * PARTS;  // chain warps
constexpr int OW = 4;          // output warps, one per lane quarter
constexpr int ST = 32 * (CW + OW + 4);  // then two warps that load V, the MMA warp and the bulk loader
constexpr int EP = C / PARTS;  // tokens of a row a chain thread has
// Registers a thread of the chain, the outputs and the rest: 4 x 88 + 88 + 40
// = 4 x 80 + 104 + 56 = 6 x 80, what the block starts with.  The compiler has 80 for
// all and spills: 36 bytes of loads at dstate 64 (52 in pieces, both scans 56), 200
// at 128 (236, 508).
template <int ND>
struct Regs {
    static constexpr int CHAIN = ND == 128 ? 88 : 80, OUT = ND == 128 ? 88 : 104, REST = ND == 128 ? 40 : 56;
};
// The MMA warp is not the scheduler's that lane quarters 0 and 1 keep busy
// (at headdim 64 the other two have nothing else to do).
constexpr int WV = CW + OW, WMMA = WV + 2, WLOAD = WV + 3;
constexpr int VT = 64;         // threads of the two warps that load V
constexpr int NV = 3;          // chunks of V in shared memory

template <int ND>
struct ScanSmem {
    static constexpr uint32_t OPS = 0, IMG = (Operands<ND>::FWD + 127) / 128 * 128, STAGE = IMG + Image::STRIDE;
    static constexpr uint32_t V0 = 2 * STAGE, VBYTES = C * 128 * 2, BYTES = V0 + NV * VBYTES;  // V on a ring of its own
};

// Tensor-memory columns: the A operands (R, and U' over it once the product
// has read R), then the accumulators S [Q; K] and R [T; X].  An MMA of 128 x 64
// takes as long as one of 128 x 128 (52 cycles against 67 as issued here), so
// the parts for the output ride along.  The state's update lies over S K,
// which is read before it is issued, and the 64 columns behind.
constexpr uint32_t COL_S = 0, COL_R = 128, COL_QS = 192, COL_KS = 256, COL_D = 256, COL_U = 384, COL_X = 448,
                   TMEM_COLS = 512;

// What the chain's threads of a row share: the largest of their first values
// and the sum of their second ones, through shared memory, two slots in turn.
// (The sum in one order, so that all of them get the same bits.)
struct RowShare {
    float2 (*slots)[PARTS * 128];
    uint64_t* bar;  // PARTS arrivals a phase, one a warp
    int* gave_up;
    int part, v, n = 0;
    __device__ __forceinline__ float2 of_all(float top, float part_of_sum) {
        float2* at = slots[n & 1];
        at[part * 128 + v] = make_float2(top, part_of_sum);
        __syncwarp();
        if (v % 32 == 0) mbar_arrive(bar);
        warp_wait(bar, n & 1, gave_up);  // (a wait that gives up leaves a wrong bound; the chunk's next wait gives up too)
        ++n;
        float2 y = at[v];
#pragma unroll
        for (int p = 1; p < PARTS; ++p) {
            const float2 x = at[p * 128 + v];
            y = make_float2(fmaxf(y.x, x.x), y.y + x.y);
        }
        return y;
    }
};

template <int NP>
__device__ __forceinline__ float top_of_pairs(const f2 (&x)[NP]) {
    float t[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        float a, b;
        un2(x[i], a, b);
        t[i & 1] = fmaxf(fmaxf(t[i & 1], fabsf(a)), fabsf(b));
    }
    return fmaxf(t[0], t[1]);
}
// Eight pairs of a lane's row, already scaled, split and stored as A-operand
// columns at `hi` and `lo`.
__device__ __forceinline__ void store_split(const f2 (&y)[8], uint32_t hi, uint32_t lo) {
    const f2 minus = mk2(-1.f, -1.f);
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, b;
        un2(y[i], a, b);
        h[i] = pack2(a, b);
        const float2 f = halves(h[i]);
        un2(fma2(mk2(f.x, f.y), minus, y[i]), a, b);
        l[i] = pack2(a, b);
    }
    tmem_st8(hi, h);
    tmem_st8(lo, l);
}

// Everything of this warp before the barrier (tensor-memory accesses too) is
// before what the barrier's waiters do.
__device__ __forceinline__ void warp_done(uint64_t* m, int lane) {
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(m);
}

// KK MMAs over the reduced dimension: A's columns 8 apart, B's descriptor STEP
// bytes (its address field, in the low word, does not carry out).
template <int KK, uint32_t STEP>
__device__ __forceinline__ void chain(uint32_t d, uint32_t a, uint64_t bd, uint32_t id, bool first) {
    const uint32_t lo = (uint32_t)bd, hi = (uint32_t)(bd >> 32);
#pragma unroll
    for (int i = 0; i < KK; ++i) mma_f16_ts(d, a + 8 * i, lo + ((i * STEP) >> 4), hi, id, !(first && i == 0));
}

// Scales of the operands made on the chain.  A half has 16 bits of exponent
// range below the point where hi and lo together lose a bit of the row's
// largest value, so a row's scale may come from a bound on it that is loose by
// up to 2^16.  With E the bound on a lane's state column, max and sum over it and
// over the chunk's tokens,
//     |R|  <= max |v| + max_i(e^{G_i} |k_i|) sqrt(N) E
//     |U'| <= max_i(|T_i|_1 e^{G_end - G_i}) |R|
//     |S+| <= e^{G_end} max |S| + max |k| sum_i |U'_i|, the next E
// (the sum as 16 times the largest of each of the lane's four threads), so no
// reduction over a row waits on the chain: an exchange between the threads of a
// row takes 290 cycles, and exact scales would want three a chunk.  The one
// exchange, of max |S| and the largest |U'|, runs beside U'^T K.  E so knows of all
// writes but the last chunk's.  Replayed on the host with random values (16 to 128
// keys, beta up to 2) U' is bounded to 2^9 .. 2^16 of its largest value.  After a
// single value 10^4 times the others, while a state of 16 keys forgets it (beta 1
// to 1.9), the last state is off by 2e-6 to 6e-6 of its largest value, fp32
// arithmetic by 3e-6 to 4e-6; with max |S| found every fourth chunk only and 64
// times the largest |U'| as the sum it was 7e-5 to 3e-4.  The exact maximum costs
// 1.4 % at 4 x 2048 x 24, 64/64 and nothing at dstate 128.
//
// What a scan's warps share beside its buffers (behind them in dynamic shared
// memory).
struct ScanShared {
    uint64_t full[2], free[2], ks, r, u, w, d, s, o, read, row[4], drain, vfull[NV], vtop[NV], vfree[NV];
    float2 sizes[2][PARTS * 128];
    float sdown[2][128], rdown[2][128], vmax[NV][128];
    uint32_t tmem;
    int gave_up;
};

template <typename E>
struct ScanArgs {
    const E* v;
    const unsigned char* image;
    const unsigned char* operands;
    const float* h0;
    E* o;
    float* h_final;
    float* states;
    float* writes;
};

// Chains on SMs.  A CTA's tensor memory fills its SM, so n chains (a head's
// scan, each a walk that cannot be split) on fewer SMs would run in whole waves:
// 192 on 152 take twice as long as 152.  Cut into `pieces` of equal length and
// run in `rounds` launches, chain i sits out rounds - pieces of them, those
// after its own, so that a round has n pieces / rounds CTAs; the state goes from
// piece to piece through `between`.  192 chains: 3 pieces in 4 rounds, forward
// 8 x 2048 x 24 64/64 in 357 us against 382 in one launch; 160: 315 against 347;
// gradients 4 x 2048 x 24 (192 chains) 536 against 550, 6 x 1024 x 16, 128/128 567
// against 574 (from a cold L2).  A round costs 10 to 18 us more than its chunks.
struct Rounds {
    int n, pieces, rounds, now;
    float* between;
    // The chain of CTA `cta` this round (or n and above: none) and its piece.
    __device__ __forceinline__ int chain(int cta, int& piece) const {
        const int s = cta % pieces, c = (now - s + rounds) % rounds, wrapped = c + pieces - rounds;
        piece = now < c ? now : now - c + max(wrapped, 0);
        return cta / pieces * rounds + c;
    }
    // Chunks before piece i of nc.
    __device__ __forceinline__ int before(int i, int nc) const { return nc * i / pieces; }
};

// KEEP = false: outputs.  KEEP = true: the state entering each chunk and the
// writes U for the gradients, no outputs.
template <typename E, int ND, bool KEEP>
__device__ __forceinline__ void scan_body(const ScanArgs<E>& g, int bh, const int* __restrict__ lens, const Shape& sh,
                                          const Rounds& turn, int piece, float* between, unsigned* status,
                                          unsigned char* smem) {
    const E* __restrict__ v = g.v;
    const unsigned char* __restrict__ image = g.image;
    const unsigned char* __restrict__ operands = g.operands;
    const float* h0 = piece > 0 ? between : g.h0;
    E* __restrict__ o = g.o;
    float* __restrict__ states = g.states;
    float* __restrict__ writes = g.writes;
    using M = ScanSmem<ND>;
    constexpr int NS = ND / PARTS;  // state elements a chain thread holds
    ScanShared& z = *reinterpret_cast<ScanShared*>(smem + M::BYTES);
    auto &mb_full = z.full, &mb_free = z.free;
    auto &mb_ks = z.ks, &mb_r = z.r, &mb_u = z.u, &mb_w = z.w, &mb_d = z.d, &mb_s = z.s, &mb_o = z.o, &mb_read = z.read;
    auto& mb_row = z.row;
    auto& mb_drain = z.drain;
    auto &mb_vfull = z.vfull, &mb_vtop = z.vtop, &mb_vfree = z.vfree;
    auto& s_sizes = z.sizes;
    auto &s_sdown = z.sdown, &s_rdown = z.rdown;
    auto& s_vtop = z.vmax;
    auto& s_tmem = z.tmem;
    auto& s_gave_up = z.gave_up;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = bh / sh.H, h = bh % sh.H, KH = sh.H / sh.G, N = sh.N, P = sh.P;
    // chunks count from this piece's first, of the sequence's `tok` and on
    const int c0 = sh.c0 + turn.before(piece, sh.c1 - sh.c0), c1 = sh.c0 + turn.before(piece + 1, sh.c1 - sh.c0);
    const int tok = c0 * C, len = max(row_len(lens, b, sh.T) - tok, 0);
    const int nck = min((len + C - 1) / C, c1 - c0);
    const int quarters = (P + 31) / 32;
    if (warp == WMMA) {
        tc::tmem_alloc(&s_tmem, TMEM_COLS);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        s_gave_up = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&mb_full[i], 1);
            tc::mbar_init(&mb_free[i], (PARTS + (KEEP ? 0 : 1)) * quarters);
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(&mb_row[i], PARTS);
        for (int i = 0; i < NV; ++i) {
            tc::mbar_init(&mb_vfull[i], VT);
            tc::mbar_init(&mb_vtop[i], quarters);
            tc::mbar_init(&mb_vfree[i], (PARTS + 1) * quarters);
        }
        tc::mbar_init(&mb_ks, 1);
        tc::mbar_init(&mb_u, 1);
        tc::mbar_init(&mb_d, 1);
        tc::mbar_init(&mb_drain, 1);
        tc::mbar_init(&mb_o, 2);
        tc::mbar_init(&mb_read, quarters);
        tc::mbar_init(&mb_r, PARTS * quarters);
        tc::mbar_init(&mb_w, PARTS * quarters);
        tc::mbar_init(&mb_s, PARTS * quarters);
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;

    if (warp < CW)
        set_registers<Regs<ND>::CHAIN, 80>();
    else if (warp < CW + OW)
        set_registers<Regs<ND>::OUT, 80>();
    else
        fewer_registers<Regs<ND>::REST>();

    if (warp < CW) {
        // ------------------------------------------------ the chain
        const int quarter = warp % 4, part = warp / 4, vc = 32 * quarter + lane;
        const bool on = vc < P;
        const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16);
        if (quarter < quarters) {
            const int64_t so = (int64_t)bh * N * P + vc;
            const int k0 = part * NS;
            f2 s[NS / 2];
#pragma unroll
            for (int i = 0; i < NS / 2; ++i) {
                const int kr = k0 + 2 * i;
                const bool there = h0 && on && kr < N;  // (N is even)
                s[i] = mk2(there ? h0[so + (int64_t)kr * P] : 0.f, there ? h0[so + (int64_t)(kr + 1) * P] : 0.f);
            }
            RowShare row{s_sizes, &mb_row[quarter], &s_gave_up, part, vc};
            auto put_state = [&](int c, float bound) {
                const RowScale sc = row_scale(bound);
                const f2 up = mk2(sc.up, sc.up);
#pragma unroll
                for (int e = 0; e < NS / 2; e += 8) {
                    f2 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = mul2(s[e + i], up);
                    store_split(y, tq + COL_S + k0 / 2 + e, tq + COL_S + ND / 2 + k0 / 2 + e);
                }
                tc::tmem_wait_st();
                if (part == 0) s_sdown[c & 1][vc] = sc.down;
                warp_done(&mb_s, lane);
                if (KEEP && on) {
                    float* dst = states + ((int64_t)bh * sh.nc + c0 + c) * N * P + vc;
#pragma unroll
                    for (int i = 0; i < NS / 2; ++i)
                        if (k0 + 2 * i < N) {
                            float a, e;
                            un2(s[i], a, e);
                            dst[(k0 + 2 * i) * P] = a;
                            dst[(k0 + 2 * i + 1) * P] = e;
                        }
                }
                return sc.down;
            };
            uint32_t vraw[EP / 2];  // this thread's tokens of V, packed as they are
            float vtop = 0.f;       // the lane's largest
            auto read_v = [&](int c) {
                const int slot = c % NV;
                if (!warp_wait(&mb_vtop[slot], c / NV & 1, &s_gave_up)) return false;
                const uint16_t* vt = reinterpret_cast<const uint16_t*>(smem + M::V0 + slot * M::VBYTES) + EP * part * P + (on ? vc : 0);
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) vraw[i] = vt[2 * i * P] | (uint32_t)vt[(2 * i + 1) * P] << 16;
                vtop = s_vtop[slot][vc];
                warp_done(&mb_vfree[slot], lane);
                return true;
            };
            float sdown = 1.f, sbound = 0.f;
            bool ok = nck > 0 && read_v(0);
            if (ok) {
                sbound = row.of_all(top_of_pairs(s), 0.f).x;
                sdown = put_state(0, sbound);
                ok = warp_wait(&mb_full[0], 0, &s_gave_up);
            }
            for (int c = 0; ok && c < nck; ++c) {
                const uint32_t ph = c & 1;
                const float* ff = reinterpret_cast<const float*>(smem + (c & 1) * M::STAGE + M::IMG + Image::F);
                f2 x[EP / 2], f[EP / 2];
                uint32_t raw[EP];
                const float rbound = fmaf(ff[Image::BND1], sbound, vtop);
                const RowScale rs = row_scale(rbound);
                auto factors = [&](int which, float m) {
#pragma unroll
                    for (int i = 0; i < EP / 4; ++i) {
                        const float4 w = *reinterpret_cast<const float4*>(ff + which + EP * part + 4 * i);
                        f[2 * i] = mul2(mk2(w.x, w.y), mk2(m, m));
                        f[2 * i + 1] = mul2(mk2(w.z, w.w), mk2(m, m));
                    }
                };
                factors(Image::KB, -sdown * rs.up);
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) {
                    const float2 w = unpack2(vraw[i], E());
                    x[i] = mul2(mk2(w.x, w.y), mk2(rs.up, rs.up));
                }
                if (part == 0) s_rdown[c & 1][vc] = rs.down;
                if (!warp_wait(&mb_ks, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                tc::tmem_ld16(tq + COL_KS + EP * part, raw);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) x[i] = fma2(f[i], raw2(raw[2 * i], raw[2 * i + 1]), x[i]);
                store_split(x, tq + COL_R + EP / 2 * part, tq + COL_R + 32 + EP / 2 * part);
                tc::tmem_wait_st();
                warp_done(&mb_r, lane);
                // while R [T; X] runs: the exact largest value of S, the next chunk's V
                const RowScale ws = row_scale(ff[Image::BND2] * rbound);
                const float top = top_of_pairs(s);
                if (c + 1 < nck && !read_v(c + 1)) break;
                factors(Image::UW, rs.down * ws.up);
                if (!warp_wait(&mb_u, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                tc::tmem_ld16(tq + COL_U + EP * part, raw);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) x[i] = mul2(f[i], raw2(raw[2 * i], raw[2 * i + 1]));
                store_split(x, tq + COL_R + EP / 2 * part, tq + COL_R + 32 + EP / 2 * part);
                tc::tmem_wait_st();
                warp_done(&mb_w, lane);
                // while U' K runs: the bound on the next state (the rows of K are scaled
                // to below 2^14, U' carries the inverse; a thread has EP of U')
                const float all = ff[Image::ALL];
                const float2 sizes = row.of_all(top, top_of_pairs(x));
                sbound = fmaf(all, sizes.x, sizes.y * ws.down * (EP * 16384.f));
                if constexpr (KEEP) {
                    if (on) {
                        float* dst = writes + (((int64_t)bh * sh.nc + c0 + c) * C + EP * part) * P + vc;
                        factors(Image::UU, rs.down);
#pragma unroll
                        for (int i = 0; i < EP / 2; ++i) {
                            float a, e;
                            un2(mul2(f[i], raw2(raw[2 * i], raw[2 * i + 1])), a, e);
                            dst[2 * i * P] = a;
                            dst[(2 * i + 1) * P] = e;
                        }
                    }
                }
                if (!warp_wait(&mb_d, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                {
                    const f2 m = mk2(ws.down, ws.down), keep = mk2(all, all);
                    uint32_t dr[NS];
#pragma unroll
                    for (int e = 0; e < NS; e += 16) tc::tmem_ld16(tq + COL_D + k0 + e, *reinterpret_cast<uint32_t(*)[16]>(dr + e));
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < NS / 2; ++i) s[i] = fma2(keep, s[i], mul2(raw2(dr[2 * i], dr[2 * i + 1]), m));
                }
                warp_done(&mb_free[c & 1], lane);
                if (c + 1 < nck) {
                    sdown = put_state(c + 1, sbound);
                    if (!warp_wait(&mb_full[(c + 1) & 1], ((c + 1) >> 1) & 1, &s_gave_up)) break;
                }
            }
            float* h_final = piece + 1 < turn.pieces ? between : g.h_final;
            if (h_final && on)
#pragma unroll
                for (int i = 0; i < NS / 2; ++i)
                    if (k0 + 2 * i < N) {
                        float a, e;
                        un2(s[i], a, e);
                        h_final[so + (int64_t)(k0 + 2 * i) * P] = a;
                        h_final[so + (int64_t)(k0 + 2 * i + 1) * P] = e;
                    }
        }
    } else if (warp < CW + OW) {
        // ------------------------------------------------ outputs
        const int quarter = warp - CW, vc = 32 * quarter + lane;
        const bool on = vc < P;
        const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16);
        // the largest |v| of a lane's column, for the chain
        auto find_top = [&](int c) {
            const int slot = c % NV;
            if (!warp_wait(&mb_vfull[slot], c / NV & 1, &s_gave_up)) return false;
            const uint16_t* vt = reinterpret_cast<const uint16_t*>(smem + M::V0 + slot * M::VBYTES) + (on ? vc : 0);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < C; ++i) m = max(m, (uint32_t)(vt[i * P] & 0x7FFF));
            s_vtop[slot][vc] = top_of<E>(m);
            warp_done(&mb_vtop[slot], lane);
            if (lane == 0) mbar_arrive(&mb_vfree[slot]);
            return true;
        };
        if (quarter < quarters && nck > 0 && find_top(0) && (nck == 1 || find_top(1))) {
            constexpr int OE = ND == 128 ? 8 : 16;  // columns at a time
            const int64_t os = (int64_t)sh.H * P;
            E* dst = KEEP ? nullptr : o + (((int64_t)b * sh.T + tok) * sh.H + h) * P + vc;
            for (int c = 0; c < nck; ++c) {
                if (c + 2 < nck && !find_top(c + 2)) break;  // (two ahead: the chain reads it a chunk early)
                if constexpr (KEEP) continue;
                unsigned char* stage = smem + (c & 1) * M::STAGE;
                if (!warp_wait(&mb_full[c & 1], (c >> 1) & 1, &s_gave_up)) break;
                if (!warp_wait(&mb_o, c & 1, &s_gave_up)) break;
                tc::fence_after_sync();
                const f2 sd = mk2(s_sdown[c & 1][vc], s_sdown[c & 1][vc]), rd = mk2(s_rdown[c & 1][vc], s_rdown[c & 1][vc]);
                const float4* coef = reinterpret_cast<const float4*>(stage + M::IMG + Image::F);
                const int n = min(len - c * C, C);
                uint32_t y[C / 2];  // the lane's 64 outputs, so that the accumulators are free before they are stored
#pragma unroll
                for (int e = 0; e < C; e += OE) {
                    uint32_t a[OE], x[OE];
                    if constexpr (OE == 16) {
                        tc::tmem_ld16(tq + COL_QS + e, a);
                        tc::tmem_ld16(tq + COL_X + e, x);
                    } else {
                        tc::tmem_ld8(tq + COL_QS + e, a);
                        tc::tmem_ld8(tq + COL_X + e, x);
                    }
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < OE; i += 4) {
                        const float4 fq = coef[(Image::OQ + e + i) / 4], fx = coef[(Image::OX + e + i) / 4];
                        const f2 lo = fma2(raw2(a[i], a[i + 1]), mul2(mk2(fq.x, fq.y), sd),
                                           mul2(raw2(x[i], x[i + 1]), mul2(mk2(fx.x, fx.y), rd)));
                        const f2 hi = fma2(raw2(a[i + 2], a[i + 3]), mul2(mk2(fq.z, fq.w), sd),
                                           mul2(raw2(x[i + 2], x[i + 3]), mul2(mk2(fx.z, fx.w), rd)));
                        y[(e + i) / 2] = pack_as<E>(lo);
                        y[(e + i) / 2 + 1] = pack_as<E>(hi);
                    }
                }
                warp_done(&mb_read, lane);
                warp_done(&mb_free[c & 1], lane);
                if (on) {
                    uint16_t* to = reinterpret_cast<uint16_t*>(dst);
                    if (n == C) {
#pragma unroll
                        for (int i = 0; i < C / 2; ++i) {
                            to[2 * i * os] = (uint16_t)y[i];
                            to[(2 * i + 1) * os] = (uint16_t)(y[i] >> 16);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < C; ++i)
                            if (i < n) to[i * os] = (uint16_t)(y[i / 2] >> (i & 1) * 16);
                    }
                }
                dst += C * os;
            }
        }
        if (!KEEP && on && sh.c0 + turn.before(piece + 1, sh.c1 - sh.c0) == sh.nc)  // behind the row's last token
            for (int t = row_len(lens, b, sh.T); t < sh.T; ++t) o[(((int64_t)b * sh.T + t) * sh.H + h) * P + vc] = from_f<E>(0.f);
    } else if (warp == WMMA) {
        // ------------------------------------------------ MMA issue
        constexpr uint32_t id64 = tc::idesc_f16(128, C), id128 = tc::idesc_f16(128, 2 * C), idn = tc::idesc_f16(128, ND);
        for (int c = 0; c < nck; ++c) {
            const uint32_t ph = c & 1;
            const uint32_t base = tc::smem_u32(smem) + (c & 1) * M::STAGE;
            const uint64_t dqk = tc::make_desc(base + M::OPS, QK<ND>::LBO, QK<ND>::SBO);
            const uint64_t dkt = tc::make_desc(base + M::OPS + Operands<ND>::KT0, KT<ND>::LBO, KT<ND>::SBO);
            const uint64_t dtx = tc::make_desc(base + M::IMG, Image::LBO, Image::SBO);
            if (!warp_wait(&mb_full[c & 1], (c >> 1) & 1, &s_gave_up)) break;
            if (!KEEP && c > 0 && !warp_wait(&mb_read, (c - 1) & 1, &s_gave_up)) break;
            if (!warp_wait(&mb_s, ph, &s_gave_up)) break;
            tc::fence_after_sync();
            const uint32_t d1 = tmem + (KEEP ? COL_KS : COL_QS), d2 = tmem + COL_U;
            const uint64_t b1 = dqk + (KEEP ? QK<ND>::KROWS >> 4 : 0);
            constexpr uint32_t id = KEEP ? id64 : id128;  // without outputs only K's and T's rows
            chain<ND / 16, 2 * QK<ND>::LBO>(d1, tmem + COL_S + ND / 2, b1, id, true);  // lo, then hi
            chain<ND / 16, 2 * QK<ND>::LBO>(d1, tmem + COL_S, b1, id, false);
            commit_elected(&mb_ks);
            if (!warp_wait(&mb_r, ph, &s_gave_up)) break;
            tc::fence_after_sync();
            chain<4, 2 * Image::LBO>(d2, tmem + COL_R + 32, dtx, id, true);  // lo hi + hi lo + hi hi
            chain<4, 2 * Image::LBO>(d2, tmem + COL_R, dtx + (Image::PART >> 4), id, false);
            chain<4, 2 * Image::LBO>(d2, tmem + COL_R, dtx, id, false);
            commit_elected(&mb_u);
            if (!KEEP) {
                commit_elected(&mb_o);
                if (lane == 0) mbar_arrive(&mb_o);  // (what the chain wrote before mb_r is before this)
            }
            if (!warp_wait(&mb_w, ph, &s_gave_up)) break;
            tc::fence_after_sync();
            chain<4, 2 * KT<ND>::LBO>(tmem + COL_D, tmem + COL_R + 32, dkt, idn, true);
            chain<4, 2 * KT<ND>::LBO>(tmem + COL_D, tmem + COL_R, dkt, idn, false);
            commit_elected(&mb_d);
        }
        if (s_gave_up) {
            commit_elected(&mb_drain);
            tc::mbar_wait_bounded(&mb_drain, 0, kDeltaWait);
        }
    } else if (warp == WLOAD) {
        // ------------------------------------------------ loader
        int last[2] = {-1, -1};  // parity of the last copies into each stage
        const unsigned char* img = image + ((int64_t)bh * sh.nc + c0) * Image::STRIDE;
        const unsigned char* ops =
            operands + (((int64_t)b * KH + h / sh.G) * sh.nc + c0) * (KEEP ? Operands<ND>::BWD : Operands<ND>::FWD);
        for (int c = 0; c < nck; ++c) {
            const uint32_t at = tc::smem_u32(smem) + (c & 1) * M::STAGE;
            if (c >= 2 && !warp_wait(&mb_free[c & 1], ((c >> 1) - 1) & 1, &s_gave_up)) break;
            if (lane == 0) {
                constexpr uint32_t from = KEEP ? QK<ND>::KROWS : 0, bytes = Operands<ND>::FWD - from;
                tc::mbar_arrive_expect_tx(&mb_full[c & 1], Image::BYTES + bytes);
                tc::bulk_g2s(at + M::OPS + from, ops + from, bytes, &mb_full[c & 1]);
                tc::bulk_g2s(at + M::IMG, img, Image::BYTES, &mb_full[c & 1]);
                last[c & 1] = (c >> 1) & 1;
                if (c + 2 < nck) {  // what the next copies into this stage read, into L2
                    prefetch_l2(ops + 2 * (KEEP ? Operands<ND>::BWD : Operands<ND>::FWD) + from, bytes);
                    prefetch_l2(img + 2 * Image::STRIDE, Image::BYTES);
                }
            }
            ops += (KEEP ? Operands<ND>::BWD : Operands<ND>::FWD);
            img += Image::STRIDE;
        }
        __syncwarp();
        if (lane == 0 && s_gave_up)  // no copy may land in shared memory that is no longer this CTA's
            for (int i = 0; i < 2; ++i)
                if (last[i] >= 0) tc::mbar_wait_bounded(&mb_full[i], last[i], kDeltaWait);
    } else {
        // ------------------------------------------------ V (rows of P elements; zeros where no token is)
        const int t = tid - 32 * WV, per = P / 8;
        for (int c = 0; c < nck; ++c) {
            const int slot = c % NV, n = min(len - c * C, C);
            const uint32_t at = tc::smem_u32(smem) + M::V0 + slot * M::VBYTES;
            const E* src = v + (((int64_t)b * sh.T + tok + (int64_t)c * C) * sh.H + h) * P;
            if (c >= NV && !warp_wait(&mb_vfree[slot], (c / NV - 1) & 1, &s_gave_up)) break;
            for (int id = t; id < C * per; id += VT) {
                const int i = id / per;
                cp_async16(at + 16 * id, src + (int64_t)min(i, n - 1) * sh.H * P + 8 * (id - i * per), i < n);
            }
            cp_async_arrive(&mb_vfull[slot]);
        }
        cp_async_wait_all();
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == WMMA) tc::tmem_dealloc(tmem, TMEM_COLS);
    if (tid == 0 && s_gave_up && status) atomicOr(status, kStatusDelta);
}

// CUT: in pieces (else the whole chain of head blockIdx.x: what a piece needs
// costs the scan registers, 1086 us against 1065 at 1 x 16384 x 32, 128/64).
template <typename E, int ND, bool CUT>
__global__ void __launch_bounds__(ST, 1) delta_scan_tc(ScanArgs<E> g, const int* __restrict__ lens, Shape sh, Rounds turn,
                                                       unsigned* status) {
    extern __shared__ __align__(1024) unsigned char smem[];
    let_next_start();  // (the next chunks' prep, on the SMs that the heads leave)
    if constexpr (CUT) {
        int piece = 0;
        const int bh = turn.chain(blockIdx.x, piece);
        if (bh < turn.n) scan_body<E, ND, false>(g, bh, lens, sh, turn, piece, turn.between, status, smem);
    } else {
        scan_body<E, ND, false>(g, blockIdx.x, lens, sh, Rounds{0, 1, 1, 0, nullptr}, 0, nullptr, status, smem);
    }
}

// --------------------------------------------------------------- backward scan
// The same walk from the last chunk, with dS in the state's place:
//     W^T  = (e^{G_end - G} K dS)^T           A = dS^T, B = K
//     Z^T  = W^T T + scale dO^T X             A = W^T, B = T^T;  A = dO^T, B = X^T
//     dS^T = e^{G_end} dS^T - (e^G beta Z)^T K + scale (e^G dO)^T Q
// The products of dO (exact in half with its row's scale in the first, split
// in the second) do not wait for the chain; four warps make their operands.
// The gradient of the state leaving each chunk is kept in `after`, Z in `zs`.
template <int ND>
struct BackSmem {
    static constexpr uint32_t K0 = 0, KT0 = QK<ND>::KROWS, QT0 = KT0 + KT<ND>::BYTES, OPS = QT0 + KT<ND>::BYTES;
    static constexpr uint32_t IMG = OPS, STAGE = IMG + Image::STRIDE;
    static constexpr uint32_t V0 = 2 * STAGE, VBYTES = C * 128 * 2, BYTES = V0 + NV * VBYTES;  // dO on a ring of its own
};
// Tensor-memory columns.  The state's update lies over K dS and T W, dO's part
// of it over dO X and dO's first operand: all read before it is issued.
namespace back {
constexpr uint32_t COL_S = 0, COL_R = 128, COL_DQ = 192, COL_KS = 256, COL_Z1 = 320, COL_D = 256, COL_Z2 = 384,
                   COL_DX = 448, COL_E = 384;
}

struct BackShared {
    uint64_t full[2], free[2], ks, r, z, w, d, s, dx, dq, row[4], drain, vfull[NV], vfree[NV];
    float2 sizes[2][PARTS * 128];
    float dxdown[128], dqdown[128], dxtop[128], dqsum[128];
    uint32_t tmem;
    int gave_up;
};

template <typename E>
struct BackArgs {
    const E* dout;
    const unsigned char* image;
    const unsigned char* operands;
    const float* dh;
    float* gh0;
    float* after;
    float* zs;
};

template <typename E, int ND>
__device__ __forceinline__ void back_scan_body(const BackArgs<E>& g, int bh, const int* __restrict__ lens, const Shape& sh,
                                               const Rounds& turn, int piece, unsigned* status, unsigned char* smem) {
    const E* __restrict__ dout = g.dout;
    const unsigned char* __restrict__ image = g.image;
    const unsigned char* __restrict__ operands = g.operands;
    const float* dh = piece > 0 ? turn.between : g.dh;
    float* __restrict__ after = g.after;
    float* __restrict__ zs = g.zs;
    using M = BackSmem<ND>;
    using namespace back;
    constexpr uint32_t COL_S = back::COL_S, COL_R = back::COL_R, COL_KS = back::COL_KS, COL_D = back::COL_D;
    constexpr int NS = ND / PARTS;
    BackShared& y = *reinterpret_cast<BackShared*>(smem + M::BYTES);
    auto &mb_full = y.full, &mb_free = y.free;
    auto &mb_ks = y.ks, &mb_r = y.r, &mb_z = y.z, &mb_w = y.w, &mb_d = y.d, &mb_s = y.s, &mb_dx = y.dx, &mb_dq = y.dq;
    auto& mb_row = y.row;
    auto& mb_drain = y.drain;
    auto &mb_vfull = y.vfull, &mb_vfree = y.vfree;
    auto& s_sizes = y.sizes;
    auto &s_dxdown = y.dxdown, &s_dqdown = y.dqdown, &s_dxtop = y.dxtop, &s_dqsum = y.dqsum;
    auto& s_tmem = y.tmem;
    auto& s_gave_up = y.gave_up;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = bh / sh.H, h = bh % sh.H, KH = sh.H / sh.G, N = sh.N, P = sh.P;
    const int len = row_len(lens, b, sh.T);
    const int first = sh.nc - turn.before(piece + 1, sh.nc);  // the row's chunks of this piece: [first, end)
    const int end = min((len + C - 1) / C, sh.nc - turn.before(piece, sh.nc)), nck = max(end - first, 0);
    const int quarters = (P + 31) / 32;
    if (warp == WMMA) {
        tc::tmem_alloc(&s_tmem, TMEM_COLS);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        s_gave_up = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&mb_full[i], 1);
            tc::mbar_init(&mb_free[i], (PARTS + 1) * quarters);
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(&mb_row[i], PARTS);
        for (int i = 0; i < NV; ++i) {
            tc::mbar_init(&mb_vfull[i], VT);
            tc::mbar_init(&mb_vfree[i], quarters);
        }
        tc::mbar_init(&mb_ks, 1);
        tc::mbar_init(&mb_z, 2);
        tc::mbar_init(&mb_d, 2);
        tc::mbar_init(&mb_drain, 1);
        tc::mbar_init(&mb_dx, quarters);
        tc::mbar_init(&mb_dq, quarters);
        tc::mbar_init(&mb_r, PARTS * quarters);
        tc::mbar_init(&mb_w, PARTS * quarters);
        tc::mbar_init(&mb_s, PARTS * quarters);
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;

    if (warp < CW)
        set_registers<Regs<ND>::CHAIN, 80>();
    else if (warp < CW + OW)
        set_registers<Regs<ND>::OUT, 80>();
    else
        fewer_registers<Regs<ND>::REST>();

    if (warp < CW) {
        // ------------------------------------------------ the chain
        const int quarter = warp % 4, part = warp / 4, vc = 32 * quarter + lane;
        const bool on = vc < P;
        const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16);
        if (quarter < quarters) {
            const int64_t so = (int64_t)bh * N * P + vc;
            const int k0 = part * NS;
            f2 s[NS / 2];
#pragma unroll
            for (int i = 0; i < NS / 2; ++i) {
                const int kr = k0 + 2 * i;
                const bool there = dh && on && kr < N;  // (N is even)
                s[i] = mk2(there ? dh[so + (int64_t)kr * P] : 0.f, there ? dh[so + (int64_t)(kr + 1) * P] : 0.f);
            }
            RowShare row{s_sizes, &mb_row[quarter], &s_gave_up, part, vc};
            auto put_state = [&](int c, float bound) {
                const RowScale sc = row_scale(bound);
                const f2 up = mk2(sc.up, sc.up);
#pragma unroll
                for (int e = 0; e < NS / 2; e += 8) {
                    f2 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = mul2(s[e + i], up);
                    store_split(y, tq + COL_S + k0 / 2 + e, tq + COL_S + ND / 2 + k0 / 2 + e);
                }
                tc::tmem_wait_st();
                warp_done(&mb_s, lane);
                if (on) {
                    float* dst = after + ((int64_t)bh * sh.nc + c) * N * P + vc;
#pragma unroll
                    for (int i = 0; i < NS / 2; ++i)
                        if (k0 + 2 * i < N) {
                            float a, e;
                            un2(s[i], a, e);
                            dst[(k0 + 2 * i) * P] = a;
                            dst[(k0 + 2 * i + 1) * P] = e;
                        }
                }
                return sc.down;
            };
            float sdown = 1.f, sbound = 0.f;
            bool ok = nck > 0;
            if (ok) {
                sbound = row.of_all(top_of_pairs(s), 0.f).x;
                sdown = put_state(end - 1, sbound);
                ok = warp_wait(&mb_full[0], 0, &s_gave_up);
            }
            for (int j = 0; ok && j < nck; ++j) {
                const int c = end - 1 - j;
                const uint32_t ph = j & 1;
                const float* ff = reinterpret_cast<const float*>(smem + (j & 1) * M::STAGE + M::IMG + Image::F);
                f2 x[EP / 2], f[EP / 2];
                uint32_t raw[EP];
                auto factors = [&](int which, float m) {
#pragma unroll
                    for (int i = 0; i < EP / 4; ++i) {
                        const float4 w = *reinterpret_cast<const float4*>(ff + which + EP * part + 4 * i);
                        f[2 * i] = mul2(mk2(w.x, w.y), mk2(m, m));
                        f[2 * i + 1] = mul2(mk2(w.z, w.w), mk2(m, m));
                    }
                };
                const float wbound = ff[Image::BND1] * sbound;
                const RowScale ws = row_scale(wbound);
                factors(Image::WK, sdown * ws.up);
                if (!warp_wait(&mb_ks, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                tc::tmem_ld16(tq + COL_KS + EP * part, raw);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) x[i] = mul2(f[i], raw2(raw[2 * i], raw[2 * i + 1]));
                store_split(x, tq + COL_R + EP / 2 * part, tq + COL_R + 32 + EP / 2 * part);
                tc::tmem_wait_st();
                warp_done(&mb_r, lane);
                // while W T runs: the exact largest value of dS
                const float top = top_of_pairs(s);
                factors(Image::ZT, ws.down);
                if (!warp_wait(&mb_z, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                tc::tmem_ld16(tq + COL_Z1 + EP * part, raw);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) x[i] = mul2(f[i], raw2(raw[2 * i], raw[2 * i + 1]));
                tc::tmem_ld16(tq + COL_Z2 + EP * part, raw);
                factors(Image::ZX, s_dxdown[vc]);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) x[i] = fma2(f[i], raw2(raw[2 * i], raw[2 * i + 1]), x[i]);
                f2 z[EP / 2];
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) z[i] = x[i];
                const RowScale rs = row_scale(fmaf(ff[Image::BND2], wbound, ff[Image::BND3] * s_dxtop[vc]));
                factors(Image::RZ, rs.up);
#pragma unroll
                for (int i = 0; i < EP / 2; ++i) x[i] = mul2(f[i], x[i]);
                store_split(x, tq + COL_R + EP / 2 * part, tq + COL_R + 32 + EP / 2 * part);
                tc::tmem_wait_st();
                warp_done(&mb_w, lane);
                if (on) {
                    float* dst = zs + (((int64_t)bh * sh.nc + c) * C + EP * part) * P + vc;
#pragma unroll
                    for (int i = 0; i < EP / 2; ++i) {
                        float a, e;
                        un2(z[i], a, e);
                        dst[2 * i * P] = a;
                        dst[(2 * i + 1) * P] = e;
                    }
                }
                // while the update runs: the bound on the next dS (the rows of K and Q
                // are scaled to below 2^14, the operands carry the inverses)
                const float all = ff[Image::ALL];
                const float2 sizes = row.of_all(top, top_of_pairs(x));
                if (!warp_wait(&mb_d, ph, &s_gave_up)) break;
                tc::fence_after_sync();
                sbound = fmaf(all, sizes.x, (sizes.y * (EP * rs.down) + s_dqsum[vc]) * 16384.f);
                {
                    const float qdown = s_dqdown[vc];
                    const f2 m = mk2(rs.down, rs.down), mq = mk2(qdown, qdown), keep = mk2(all, all);
#pragma unroll
                    for (int e = 0; e < NS; e += 16) {
                        tc::tmem_ld16(tq + COL_D + k0 + e, raw);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            s[e / 2 + i] = fma2(keep, s[e / 2 + i], mul2(raw2(raw[2 * i], raw[2 * i + 1]), m));
                        tc::tmem_ld16(tq + COL_E + k0 + e, raw);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            s[e / 2 + i] = fma2(raw2(raw[2 * i], raw[2 * i + 1]), mq, s[e / 2 + i]);
                    }
                }
                warp_done(&mb_free[j & 1], lane);
                if (j + 1 < nck) {
                    sdown = put_state(c - 1, sbound);
                    if (!warp_wait(&mb_full[(j + 1) & 1], ((j + 1) >> 1) & 1, &s_gave_up)) break;
                }
            }
            float* gh0 = piece + 1 < turn.pieces ? turn.between : g.gh0;
            if (gh0 && on)
#pragma unroll
                for (int i = 0; i < NS / 2; ++i)
                    if (k0 + 2 * i < N) {
                        float a, e;
                        un2(s[i], a, e);
                        gh0[so + (int64_t)(k0 + 2 * i) * P] = a;
                        gh0[so + (int64_t)(k0 + 2 * i + 1) * P] = e;
                    }
        }
    } else if (warp < CW + OW) {
        // ------------------------------------------------ dO's operands
        const int quarter = warp - CW, vc = 32 * quarter + lane;
        const bool on = vc < P;
        const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16);
        if (quarter < quarters) {
            for (int j = 0; j < nck; ++j) {
                const int slot = j % NV;
                if (!warp_wait(&mb_vfull[slot], j / NV & 1, &s_gave_up)) break;
                const uint16_t* dt = reinterpret_cast<const uint16_t*>(smem + M::V0 + slot * M::VBYTES) + (on ? vc : 0);
                uint32_t raw[C / 2];
#pragma unroll
                for (int i = 0; i < C / 2; ++i) raw[i] = dt[2 * i * P] | (uint32_t)dt[(2 * i + 1) * P] << 16;
                if (!on)
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) raw[i] = 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&mb_vfree[slot]);
                if (!warp_wait(&mb_full[j & 1], (j >> 1) & 1, &s_gave_up)) break;
                const float* ff = reinterpret_cast<const float*>(smem + (j & 1) * M::STAGE + M::IMG + Image::F);
                uint32_t m = 0;
                float qt = 0.f, qsum = 0.f;
#pragma unroll
                for (int i = 0; i < C / 2; ++i) {
                    m = __vmaxu2(m, raw[i] & 0x7FFF7FFFu);
                    const float2 w = unpack2(raw[i], E()), f = *reinterpret_cast<const float2*>(ff + Image::DQ + 2 * i);
                    const float a = fabsf(w.x * f.x), b = fabsf(w.y * f.y);
                    qt = fmaxf(fmaxf(qt, a), b);
                    qsum += a + b;
                }
                const float top = top_of<E>(m);
                const RowScale xs = row_scale(top), qs = row_scale(qt);
                // the columns are free once the chain has stored the state (it has read what lay there)
                if (!warp_wait(&mb_s, j & 1, &s_gave_up)) break;
                tc::fence_after_sync();
                s_dxdown[vc] = xs.down;
                s_dxtop[vc] = top;
                s_dqdown[vc] = qs.down;
                s_dqsum[vc] = qsum;
#pragma unroll
                for (int e = 0; e < C / 2; e += 8) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 y = unpack2(raw[e + i], E());
                        w[i] = pack2(y.x * xs.up, y.y * xs.up);
                    }
                    tmem_st8(tq + COL_DX + e, w);
                }
                tc::tmem_wait_st();
                warp_done(&mb_dx, lane);
#pragma unroll
                for (int e = 0; e < C / 2; e += 8) {
                    f2 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 w = unpack2(raw[e + i], E()), f = *reinterpret_cast<const float2*>(ff + Image::DQ + 2 * (e + i));
                        y[i] = mul2(mk2(w.x * f.x, w.y * f.y), mk2(qs.up, qs.up));
                    }
                    store_split(y, tq + COL_DQ + e, tq + COL_DQ + 32 + e);
                }
                tc::tmem_wait_st();
                warp_done(&mb_dq, lane);
                if (lane == 0) mbar_arrive(&mb_free[j & 1]);
            }
        }
    } else if (warp == WMMA) {
        // ------------------------------------------------ MMA issue
        constexpr uint32_t id64 = tc::idesc_f16(128, C), idn = tc::idesc_f16(128, ND);
        for (int j = 0; j < nck; ++j) {
            const uint32_t ph = j & 1;
            const uint32_t base = tc::smem_u32(smem) + (j & 1) * M::STAGE;
            const uint64_t dk = tc::make_desc(base + M::K0, QK<ND>::LBO, QK<ND>::SBO);
            const uint64_t dkt = tc::make_desc(base + M::KT0, KT<ND>::LBO, KT<ND>::SBO);
            const uint64_t dqt = tc::make_desc(base + M::QT0, KT<ND>::LBO, KT<ND>::SBO);
            const uint64_t dtt = tc::make_desc(base + M::IMG, Image::LBO, Image::SBO);
            const uint64_t dxt = dtt + ((8 * Image::SBO) >> 4);
            if (!warp_wait(&mb_full[j & 1], (j >> 1) & 1, &s_gave_up)) break;
            if (!warp_wait(&mb_s, ph, &s_gave_up)) break;
            tc::fence_after_sync();
            chain<ND / 16, 2 * QK<ND>::LBO>(tmem + COL_KS, tmem + COL_S + ND / 2, dk, id64, true);  // lo, then hi
            chain<ND / 16, 2 * QK<ND>::LBO>(tmem + COL_KS, tmem + COL_S, dk, id64, false);
            commit_elected(&mb_ks);
            if (!warp_wait(&mb_dx, ph, &s_gave_up)) break;
            tc::fence_after_sync();
            chain<4, 2 * Image::LBO>(tmem + COL_Z2, tmem + COL_DX, dxt + (Image::PART >> 4), id64, true);
            chain<4, 2 * Image::LBO>(tmem + COL_Z2, tmem + COL_DX, dxt, id64, false);
            if (!warp_wait(&mb_r, ph, &s_gave_up)) break;
            tc::fence_after_sync();
            chain<4, 2 * Image::LBO>(tmem + COL_Z1, tmem + COL_R + 32, dtt, id64, true);  // lo hi + hi lo + hi hi
            chain<4, 2 * Image::LBO>(tmem + COL_Z1, tmem + COL_R, dtt + (Image::PART >> 4), id64, false);
            chain<4, 2 * Image::LBO>(tmem + COL_Z1, tmem + COL_R, dtt, id64, false);
            commit_elected(&mb_z);
            if (lane == 0) mbar_arrive(&mb_z);  // (dO's scales, written before mb_dx, are before this)
            if (!warp_wait(&mb_w, ph, &s_gave_up)) break;
            if (!warp_wait(&mb_dq, ph, &s_gave_up)) break;
            tc::fence_after_sync();
            chain<4, 2 * KT<ND>::LBO>(tmem + COL_D, tmem + COL_R + 32, dkt, idn, true);
            chain<4, 2 * KT<ND>::LBO>(tmem + COL_D, tmem + COL_R, dkt, idn, false);
            chain<4, 2 * KT<ND>::LBO>(tmem + COL_E, tmem + COL_DQ + 32, dqt, idn, true);
            chain<4, 2 * KT<ND>::LBO>(tmem + COL_E, tmem + COL_DQ, dqt, idn, false);
            commit_elected(&mb_d);
            if (lane == 0) mbar_arrive(&mb_d);
        }
        if (s_gave_up) {
            commit_elected(&mb_drain);
            tc::mbar_wait_bounded(&mb_drain, 0, kDeltaWait);
        }
    } else if (warp == WLOAD) {
        // ------------------------------------------------ loader
        int last[2] = {-1, -1};  // parity of the last copies into each stage
        const unsigned char* img = image + (int64_t)bh * sh.nc * Image::STRIDE;
        const unsigned char* ops = operands + ((int64_t)b * KH + h / sh.G) * sh.nc * Operands<ND>::BWD + QK<ND>::KROWS;
        for (int j = 0; j < nck; ++j) {
            const int c = end - 1 - j;
            const uint32_t at = tc::smem_u32(smem) + (j & 1) * M::STAGE;
            if (j >= 2 && !warp_wait(&mb_free[j & 1], ((j >> 1) - 1) & 1, &s_gave_up)) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&mb_full[j & 1], Image::BYTES + M::OPS);
                tc::bulk_g2s(at + M::K0, ops + (int64_t)c * Operands<ND>::BWD, M::OPS, &mb_full[j & 1]);
                tc::bulk_g2s(at + M::IMG, img + (int64_t)c * Image::STRIDE, Image::BYTES, &mb_full[j & 1]);
                last[j & 1] = (j >> 1) & 1;
                if (c - 2 >= first) {  // what the next copies into this stage read, into L2
                    prefetch_l2(ops + (int64_t)(c - 2) * Operands<ND>::BWD, M::OPS);
                    prefetch_l2(img + (int64_t)(c - 2) * Image::STRIDE, Image::BYTES);
                }
            }
        }
        __syncwarp();
        if (lane == 0 && s_gave_up)  // no copy may land in shared memory that is no longer this CTA's
            for (int i = 0; i < 2; ++i)
                if (last[i] >= 0) tc::mbar_wait_bounded(&mb_full[i], last[i], kDeltaWait);
    } else {
        // ------------------------------------------------ dO (rows of P elements; zeros where no token is)
        const int t = tid - 32 * WV, per = P / 8;
        for (int j = 0; j < nck; ++j) {
            const int c = end - 1 - j, slot = j % NV, n = min(len - c * C, C);
            const uint32_t at = tc::smem_u32(smem) + M::V0 + slot * M::VBYTES;
            const E* src = dout + (((int64_t)b * sh.T + (int64_t)c * C) * sh.H + h) * P;
            if (j >= NV && !warp_wait(&mb_vfree[slot], (j / NV - 1) & 1, &s_gave_up)) break;
            for (int id = t; id < C * per; id += VT) {
                const int i = id / per;
                cp_async16(at + 16 * id, src + (int64_t)min(i, n - 1) * sh.H * P + 8 * (id - i * per), i < n);
            }
            cp_async_arrive(&mb_vfull[slot]);
        }
        cp_async_wait_all();
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == WMMA) tc::tmem_dealloc(tmem, TMEM_COLS);
    if (tid == 0 && s_gave_up && status) atomicOr(status, kStatusDelta);
}

// Both of the gradients' scans, which do not need one another, in one launch a
// round: chains 0 .. n / 2 - 1 run the backward scan, the others the forward.
template <typename E, int ND>
__global__ void __launch_bounds__(ST, 1) delta_both_scans_tc(BackArgs<E> back, ScanArgs<E> fwd, const int* __restrict__ lens,
                                                             Shape sh, Rounds turn, unsigned* status) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const int heads = turn.n / 2;
    int piece = 0;
    const int i = turn.chain(blockIdx.x, piece);
    if (i < heads)
        back_scan_body<E, ND>(back, i, lens, sh, turn, piece, status, smem);
    else if (i < turn.n)
        scan_body<E, ND, true>(fwd, i - heads, lens, sh, turn, piece, turn.between + (int64_t)heads * sh.N * sh.P, status,
                               smem);
}

// --------------------------------------------------------------- dQ, dK, dV, dg, dbeta
// One CTA per chunk and value head (the formulas stand at the head of
// delta.cu), the products on the tensor cores with tokens i in the lanes: row
// i of what becomes dQ in lane i, of dK in lane 64 + i, so that
//     [dO; Z] U^T, [Q; K] K^T          64 columns each
//     [dO; Z] S^T, [Z; U] dS^T         N columns each (the first rows of the
//                                      second are not used)
//     [Pm 0; W + W^T  Pm^T] [K; Q]     N columns
// take five MMA chains of 128 rows.  S, dS, Z and U are fp32 and are split on
// the way into shared memory, a row a scale; dO is exact with its scale, Pm
// and W are split with one scale a chunk (into tensor memory, over the first
// two products).  4 x 2048 x 24, 64/64: 211 us for 406 MB read, 2 TB/s; bound by
// the latency of a CTA's stages (20 us from its loads to its last store, issue 27 %
// busy) at the two CTAs an SM that 128 registers a thread leave.  512 threads a
// CTA took 246 us against 228 then, an L2 prefetch of the next CTAs' data 236.
template <int ND, int PD>
struct GradSmem {
    static constexpr int NT = ND == 128 ? 512 : 256;  // 32 columns of dQ, dK a thread
    static constexpr uint32_t LBO = 128, SBO = (PD / 8) * LBO, ROWS = 8 * SBO;  // 64 rows
    static constexpr uint32_t HI = 0, LO = 3 * ROWS, ST = 6 * ROWS, STP = (ND / 8) * SBO;  // [dO; Z; U], their rests; S
    // The operands of K and Q; at the widest, where not everything fits, K^T and
    // Q^T come late, over dO (read by then) and its rest.
    static constexpr bool LATE = ND == 128 && PD == 128;
    static constexpr uint32_t OPS = ST + 2 * STP;
    // Pm below the diagonal and W^T above, fp32, over Q and K when those are
    // read: 65 columns a row, so that neither a row's nor a column's readers
    // meet in a bank.
    static constexpr int LM = C + 1;
    static constexpr uint32_t MAT = OPS, MAT_BYTES = (4 * C * LM + 127) / 128 * 128;
    static constexpr uint32_t QK_BYTES = QK<ND>::BYTES > MAT_BYTES ? QK<ND>::BYTES : MAT_BYTES;
    static constexpr uint32_t KT0 = LATE ? HI : OPS + QK_BYTES, QT0 = LATE ? LO : KT0 + KT<ND>::BYTES;
    static constexpr uint32_t BYTES = OPS + QK_BYTES + (LATE ? 0 : 2 * KT<ND>::BYTES);
    static_assert(!LATE || KT<ND>::BYTES <= ROWS, "K^T over dO");
};

// 8 rows a warp (row lane % 8), a lane's column groups lane / 8, + 4, ..: the
// rows of an fp32 matrix with `width` columns, zeros past them.
template <int NG>
__device__ __forceinline__ void load_groups(float (&x)[NG][8], const float* row, int lane, int width, bool there) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int c = 8 * (lane / 8 + 4 * g);
        const bool in = there && c < width;
        const float4 a = in ? __ldcs(reinterpret_cast<const float4*>(row + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 b = in ? __ldcs(reinterpret_cast<const float4*>(row + c + 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[g][0] = a.x, x[g][1] = a.y, x[g][2] = a.z, x[g][3] = a.w;
        x[g][4] = b.x, x[g][5] = b.y, x[g][6] = b.z, x[g][7] = b.w;
    }
}
// The largest of a row over its four lanes.
__device__ __forceinline__ float over_row(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
// The groups scaled by their row's power of two, split and stored; returns
// the inverse scale.
template <int NG>
__device__ __forceinline__ float store_groups(const float (&x)[NG][8], unsigned char* hi, unsigned char* lo, int lane) {
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int u = 0; u < 8; ++u) top = fmaxf(top, fabsf(x[g][u]));
    const RowScale s = row_scale(over_row(top));
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) split2(x[g][2 * u] * s.up, x[g][2 * u + 1] * s.up, h[u], l[u]);
        const uint32_t at = (lane / 8 + 4 * g) * 128 + (lane % 8) * 16;
        *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
    return s.down;
}

template <typename E, typename O, int ND, int PD>
__global__ void __launch_bounds__(GradSmem<ND, PD>::NT, ND == 128 || PD == 128 ? 1 : 2)
    delta_grad_tc(const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v, const E* __restrict__ dout,
                  const float* __restrict__ g, const float* __restrict__ beta, const int* __restrict__ lens, float scale,
                  const unsigned char* __restrict__ image_t, const unsigned char* __restrict__ operands,
                  const float* __restrict__ states, const float* __restrict__ after, const float* __restrict__ writes,
                  const float* __restrict__ zs, O* __restrict__ gq, O* __restrict__ gk, E* __restrict__ gv,
                  float* __restrict__ gg, float* __restrict__ gbeta, Shape sh, unsigned* status) {
    using M = GradSmem<ND, PD>;
    constexpr int NT = M::NT, NW = NT / 32, NPART = NT / 128, CJ = C / NPART, NG = PD / 32;
    constexpr uint32_t COL_DU = 0, COL_KK = 64, COL_S = 128, COL_D = 128 + ND, COLS = ND == 128 ? 512 : 256;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(16) Decays d;
    __shared__ __align__(16) DecayTables tab;
    __shared__ __align__(16) float s_kd[C], s_qd[C], s_u[C], s_rows[2 * C], s_st[ND], s_ds[ND];
    __shared__ float s_zv[C], s_gb[NPART][C], s_qgq[NPART][C], s_kz[NPART][C], s_top[NW], s_kus[NW], s_kqd;
    __shared__ double s_dot[NW];
    __shared__ __align__(8) uint64_t mb_ops, mb_late, mb_1, mb_2, mb_3, mb_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_gave_up;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x % sh.nc, bh = blockIdx.x / sh.nc;
    const int b = bh / sh.H, h = bh % sh.H, KH = sh.H / sh.G, N = sh.N, P = sh.P;
    const int len = row_len(lens, b, sh.T), n = min(len - c * C, C), here = min(sh.T - c * C, C);
    const int64_t t0 = (int64_t)b * sh.T + (int64_t)c * C, ci = (int64_t)bh * sh.nc + c;
    const int64_t ko = (t0 * KH + h / sh.G) * N, ks = (int64_t)KH * N, vo = (t0 * sh.H + h) * P, vs = (int64_t)sh.H * P;
    const int64_t go = (t0 * sh.H + h) * N, gs = (int64_t)sh.H * N;  // of gq and gk: the same as ko when G = 1
    if (n < here) {  // tokens that are not there
        const int from = max(n, 0);
        for (int e = tid; e < (here - from) * N; e += NT) {
            gq[go + (from + e / N) * gs + e % N] = from_f<O>(0.f);
            gk[go + (from + e / N) * gs + e % N] = from_f<O>(0.f);
        }
        for (int e = tid; e < (here - from) * P; e += NT) gv[vo + (from + e / P) * vs + e % P] = from_f<E>(0.f);
        for (int i = from + tid; i < here; i += NT) gg[(t0 + i) * sh.H + h] = gbeta[(t0 + i) * sh.H + h] = 0.f;
    }
    if (n <= 0) return;
    const unsigned char* ops = operands + (((int64_t)b * KH + h / sh.G) * sh.nc + c) * Operands<ND>::BWD;
    if (warp == 0) {
        tc::tmem_alloc(&s_tmem, COLS);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        s_gave_up = 0;
        tab.steep = 0;
        tc::mbar_init(&mb_ops, 1);
        tc::mbar_init(&mb_1, 1);
        tc::mbar_init(&mb_2, 1);
        tc::mbar_init(&mb_3, 2);
        tc::mbar_init(&mb_late, 1);
        tc::mbar_init(&mb_drain, 1);
        tc::mbar_fence_init();
        tc::mbar_arrive_expect_tx(&mb_ops, M::LATE ? QK<ND>::BYTES : Operands<ND>::BWD);
        tc::bulk_g2s(tc::smem_u32(smem + M::OPS), ops, QK<ND>::BYTES, &mb_ops);
        if (!M::LATE) tc::bulk_g2s(tc::smem_u32(smem + M::KT0), ops + Operands<ND>::KT0, 2 * KT<ND>::BYTES, &mb_ops);
    }
    // Z (with dV and z.v), U, dO: 8 rows a warp, all loads before the first use
    const int rg = warp % 8, ti = 8 * rg + lane % 8, srow = 8 * warp + lane % 8;
    const bool has_z = NW == 8 || warp < 8, has_u = NW == 8 || warp >= 8;  // dO goes with Z
    float zx[NG][8], ux[NG][8], sx[NG][8];
    uint4 dr[NG], vr[NG];
    float bt = 0.f;
    if (has_z) {
        load_groups<NG>(zx, zs + (ci * C + ti) * P, lane, P, true);
        const int64_t row = vo + ti * vs;
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const int col = 8 * (lane / 8 + 4 * e);
            const bool in = ti < n && col < P;
            dr[e] = in ? *reinterpret_cast<const uint4*>(dout + row + col) : make_uint4(0, 0, 0, 0);
            vr[e] = in ? *reinterpret_cast<const uint4*>(v + row + col) : make_uint4(0, 0, 0, 0);
        }
        if (ti < n) bt = beta[(t0 + ti) * sh.H + h];
    }
    if (has_u) load_groups<NG>(ux, writes + (ci * C + ti) * P, lane, P, true);
    load_groups<NG>(sx, states + (ci * N + srow) * P, lane, P, srow < N);
    if (warp == NW - 1) chunk_decays(d, g + t0 * sh.H + h, beta + t0 * sh.H + h, sh.H, n, lane);
    if (tid < C) {
        const float* fb = reinterpret_cast<const float*>(image_t + ci * Image::STRIDE + Image::F);
        s_kd[tid] = fb[Image::KD + tid];
        s_qd[tid] = fb[Image::QD + tid];
    }
    unsigned char* hi = smem + M::HI + rg * M::SBO;
    if (has_z) {
        const float down = store_groups<NG>(zx, hi + M::ROWS, hi + 4 * M::ROWS, lane);
        if (lane < 8) s_rows[C + ti] = down;
        float zv = 0.f;
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const uint32_t in[4] = {vr[e].x, vr[e].y, vr[e].z, vr[e].w};
            uint32_t out[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 y = unpack2(in[u], E());
                zv = fmaf(y.x, zx[e][2 * u], fmaf(y.y, zx[e][2 * u + 1], zv));
                out[u] = pack_as<E>(mk2(bt * zx[e][2 * u], bt * zx[e][2 * u + 1]));
            }
            const int col = 8 * (lane / 8 + 4 * e);
            if (ti < n && col < P) *reinterpret_cast<uint4*>(gv + vo + ti * vs + col) = make_uint4(out[0], out[1], out[2], out[3]);
            m = __vmaxu2(m, __vmaxu2(absmax2(dr[e].x, dr[e].y), absmax2(dr[e].z, dr[e].w)));
        }
        zv += __shfl_xor_sync(0xffffffffu, zv, 8);
        zv += __shfl_xor_sync(0xffffffffu, zv, 16);
        const RowScale sc = row_scale(over_row(top_of<E>(m)));
        if (lane < 8) {
            s_zv[ti] = zv;
            s_rows[ti] = sc.down;
        }
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const uint32_t in[4] = {dr[e].x, dr[e].y, dr[e].z, dr[e].w};
            uint32_t out[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 y = unpack2(in[u], E());
                out[u] = pack2(y.x * sc.up, y.y * sc.up);
            }
            const uint32_t at = (lane / 8 + 4 * e) * 128 + (lane % 8) * 16;
            *reinterpret_cast<uint4*>(hi + at) = make_uint4(out[0], out[1], out[2], out[3]);
            *reinterpret_cast<uint4*>(hi + 3 * M::ROWS + at) = make_uint4(0, 0, 0, 0);
        }
    }
    if (has_u) {
        const float down = store_groups<NG>(ux, hi + 2 * M::ROWS, hi + 5 * M::ROWS, lane);
        if (lane < 8) s_u[ti] = down;
    }
    // S into its operand; dS into registers for the same place later, and <S, dS>
    float ds[NG][8];
    {
        static_assert(NW * 8 == ND, "a warp has 8 rows of the state");
        load_groups<NG>(ds, after + (ci * N + srow) * P, lane, P, srow < N);
        const float down = store_groups<NG>(sx, smem + M::ST + warp * M::SBO, smem + M::ST + M::STP + warp * M::SBO, lane);
        if (lane < 8) s_st[srow] = down;
    }
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem, base = tc::smem_u32(smem);
    constexpr uint32_t id64 = tc::idesc_f16(128, C), idn = tc::idesc_f16(128, ND);
    // a (128 rows, hi and their rests) times b: lo hi + hi lo + hi hi
    auto split_product = [&](uint32_t dcol, uint32_t a, uint32_t bb, uint32_t brest, uint32_t id) {
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint64_t da = tc::make_desc(base + a + (p == 0 ? 3 * M::ROWS : 0), M::LBO, M::SBO);
            const uint64_t db = tc::make_desc(base + bb + (p == 1 ? brest : 0), M::LBO, M::SBO);
#pragma unroll
            for (int kk = 0; kk < PD / 16; ++kk)
                tc::mma_f16(tmem + dcol, da + 16 * kk, db + 16 * kk, id, p || kk);
        }
    };
    if (tid == 0) {
        wait_or_give_up(&mb_ops, 0, &s_gave_up);
        split_product(COL_DU, M::HI, M::HI + 2 * M::ROWS, 3 * M::ROWS, id64);
        const uint64_t dqk = tc::make_desc(base + M::OPS, QK<ND>::LBO, QK<ND>::SBO);
#pragma unroll
        for (int kk = 0; kk < ND / 16; ++kk)
            tc::mma_f16(tmem + COL_KK, dqk + 16 * kk, dqk + (QK<ND>::KROWS >> 4) + 16 * kk, id64, kk != 0);
        tc::commit(&mb_1);
        split_product(COL_S, M::HI, M::ST, M::STP, idn);
        tc::commit(&mb_2);
    }
    __syncwarp();
    if (tid < 256) decay_tables(tab, d, s_u, tid);  // (with U's scales, which go with them)
    {
        float part = 0.f;
#pragma unroll
        for (int e = 0; e < NG; ++e)
#pragma unroll
            for (int u = 0; u < 8; ++u) part = fmaf(sx[e][u], ds[e][u], part);
        double dot = (double)part;
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) s_dot[warp] = dot;
    }
    if (warp == NW - 1) {  // the largest of K's and Q's inverse scales
        float m = fmaxf(fmaxf(s_kd[lane], s_kd[lane + 32]), fmaxf(s_qd[lane], s_qd[lane + 32]));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) s_kqd = m;
    }
    __syncthreads();

    // ---- Pm and W: row i of Pm in the lanes of dQ, of W in those of dK
    const int quarter = warp % 4, part = warp / 4, row = 32 * quarter + lane, i = row % C, j0 = CJ * part;
    const bool is_k = quarter >= 2;
    const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16);
    float* mat = reinterpret_cast<float*>(smem + M::MAT);
    float* mrow = mat + i * M::LM;  // row i
    float* mcol = mat + i;          // column i
    const bool above = 32 * (quarter % 2) + 31 < j0;                  // every pair of this warp has i < j
    warp_wait(&mb_1, 0, &s_gave_up);
    tc::fence_after_sync();
    {
        float top = 0.f, gb = 0.f;
        if (!above) {
            const float ri = s_rows[row] * (is_k ? 1.f : scale), re = ri * tab.e[i], nb = -d.beta[i];
            const int last = is_k ? i - 1 : i;
            const bool steep = tab.steep;
            // eight columns; MASK where some of the warp's rows end among them
            auto columns = [&](int j, auto mask) {
                constexpr bool MASK = decltype(mask)::value;
                uint32_t du[8], kk[8];
                tc::tmem_ld8(tq + COL_DU + j, du);
                if (is_k) tc::tmem_ld8(tq + COL_KK + j, kk);
                tc::tmem_wait_ld();
                float x[8];
                if (!steep) {
#pragma unroll
                    for (int u = 0; u < 8; u += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(tab.f[i / 16] + j + u);
                        x[u] = __uint_as_float(du[u]) * (re * f.x), x[u + 1] = __uint_as_float(du[u + 1]) * (re * f.y);
                        x[u + 2] = __uint_as_float(du[u + 2]) * (re * f.z), x[u + 3] = __uint_as_float(du[u + 3]) * (re * f.w);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 8; ++u) x[u] = __uint_as_float(du[u]) * (ri * s_u[j + u]) * steep_decay(d, i, j + u);
                }
                if (MASK)
#pragma unroll
                    for (int u = 0; u < 8; ++u) x[u] = j + u <= last ? x[u] : 0.f;
                if (is_k) {
#pragma unroll
                    for (int u = 0; u < 8; u += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(s_kd + j + u);
                        const float fu[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const float y = __uint_as_float(kk[u + w]) * fu[w];
                            // (by select: nothing above the diagonal may reach the sum)
                            gb = fmaf(x[u + w], !MASK || j + u + w <= last ? y : 0.f, gb);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        x[u] *= nb;
                        if (!MASK || j + u <= last) mcol[(j + u) * M::LM] = x[u];
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        if (!MASK || j + u <= last) mrow[j + u] = x[u];
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) top = fmaxf(top, fabsf(x[u]));
            };
#pragma unroll 1
            for (int j = j0; j < j0 + CJ; j += 8) {
                if (j + 8 <= 32 * (quarter % 2))
                    columns(j, std::false_type());
                else
                    columns(j, std::true_type());
            }
        }
        // sum_j W_ij k_i.k_j = -beta_i times what dbeta wants
        if (is_k) s_gb[part][i] = gb * s_kd[i];
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) s_top[warp] = top;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    float top = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, s_top[w]);
    const RowScale ps = row_scale(top * s_kqd);
    // the A operand of the last product: [Pm 0; W + W^T  Pm^T], times the inverse scales of K and Q
#pragma unroll 1
    for (int e = 0; e < CJ; e += 16) {
        const int j = j0 + e;
        f2 a[8];
        const f2 up = mk2(ps.up, ps.up);
        const float *row0 = mrow + j, *col0 = mcol + j * M::LM;
        if (is_k) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {  // W below the diagonal lies at (column, row), above it at (row, column)
                float x[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int cc = 2 * u + w;
                    x[w] = *(j + cc < i ? col0 + cc * M::LM : row0 + cc);
                    if (j + cc == i) x[w] = 0.f;
                }
                a[u] = mul2(mul2(mk2(x[0], x[1]), *reinterpret_cast<const f2*>(s_kd + j + 2 * u)), up);
            }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                float x[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) x[w] = j + 2 * u + w <= i ? row0[2 * u + w] : 0.f;
                a[u] = mul2(mul2(mk2(x[0], x[1]), *reinterpret_cast<const f2*>(s_kd + j + 2 * u)), up);
            }
        }
        store_split(a, tq + j / 2, tq + 32 + j / 2);
        if (is_k) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                float x[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) x[w] = j + 2 * u + w >= i ? col0[(2 * u + w) * M::LM] : 0.f;
                a[u] = mul2(mul2(mk2(x[0], x[1]), *reinterpret_cast<const f2*>(s_qd + j + 2 * u)), up);
            }
            store_split(a, tq + 64 + j / 2, tq + 96 + j / 2);
        } else {
            const uint32_t zero[8] = {};
            tmem_st8(tq + 64 + j / 2, zero);
            tmem_st8(tq + 96 + j / 2, zero);
        }
    }
    tc::tmem_wait_st();

    // ---- the products with S; dS in its place
    constexpr int NC = ND / NPART;  // 32
    const int n0 = NC * part;
    float first[NC];  // of dQ: its part from S; of dK: -beta e^G Z S^T
    float kz = 0.f, kus = 0.f, qgq = 0.f;
    uint4 own[NC / 8];  // q's row for dQ, k's for dK
    {
        const E* src = (is_k ? k : q) + ko + i * ks + n0;
#pragma unroll
        for (int e = 0; e < NC / 8; ++e)
            own[e] = i < n && n0 + 8 * e < N ? *reinterpret_cast<const uint4*>(src + 8 * e) : make_uint4(0, 0, 0, 0);
        uint32_t r[NC];
        warp_wait(&mb_2, 0, &s_gave_up);
        tc::fence_after_sync();
        tmem_ld32(tq + COL_S + n0, r);
        tc::tmem_wait_ld();
        const float f = s_rows[row] * (is_k ? 1.f : scale * d.in[i]), bg = is_k ? -d.beta[i] * d.in[i] : 1.f;
#pragma unroll
        for (int e = 0; e < NC; e += 4) {
            const float4 w = *reinterpret_cast<const float4*>(s_st + n0 + e);
            first[e] = __uint_as_float(r[e]) * (f * w.x), first[e + 1] = __uint_as_float(r[e + 1]) * (f * w.y);
            first[e + 2] = __uint_as_float(r[e + 2]) * (f * w.z), first[e + 3] = __uint_as_float(r[e + 3]) * (f * w.w);
        }
        if (is_k) {
#pragma unroll
            for (int e = 0; e < NC; e += 2) {
                const float2 y = unpack2(reinterpret_cast<const uint32_t*>(&own[e / 8])[e % 8 / 2], E());
                kz = fmaf(y.x, first[e], fmaf(y.y, first[e + 1], kz));
                first[e] *= bg;
                first[e + 1] *= bg;
            }
        }
        const float down = store_groups<NG>(ds, smem + M::ST + warp * M::SBO, smem + M::ST + M::STP + warp * M::SBO, lane);
        if (lane < 8) s_ds[srow] = down;
    }
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) {
        if (lane == 0) {
            if (M::LATE) {
                tc::mbar_arrive_expect_tx(&mb_late, 2 * KT<ND>::BYTES);
                tc::bulk_g2s(base + M::KT0, ops + Operands<ND>::KT0, KT<ND>::BYTES, &mb_late);
                tc::bulk_g2s(base + M::QT0, ops + Operands<ND>::QT0, KT<ND>::BYTES, &mb_late);
            }
            split_product(COL_D, M::HI + M::ROWS, M::ST, M::STP, idn);
            tc::commit(&mb_3);
        }
        __syncwarp();
        if (M::LATE) warp_wait(&mb_late, 0, &s_gave_up);
        const uint64_t dkt = tc::make_desc(base + M::KT0, KT<ND>::LBO, KT<ND>::SBO);
        const uint64_t dqt = tc::make_desc(base + M::QT0, KT<ND>::LBO, KT<ND>::SBO);
        chain<4, 2 * KT<ND>::LBO>(tmem + COL_S, tmem + 32, dkt, idn, true);
        chain<4, 2 * KT<ND>::LBO>(tmem + COL_S, tmem + 96, dqt, idn, false);
        chain<4, 2 * KT<ND>::LBO>(tmem + COL_S, tmem, dkt, idn, false);
        chain<4, 2 * KT<ND>::LBO>(tmem + COL_S, tmem + 64, dqt, idn, false);
        commit_elected(&mb_3);
    }
    warp_wait(&mb_3, 0, &s_gave_up);
    tc::fence_after_sync();
    {
        uint32_t r[NC];
        tmem_ld32(tq + COL_S + n0, r);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < NC; ++e) first[e] = fmaf(__uint_as_float(r[e]), ps.down, first[e]);
        if (is_k) {
            tmem_ld32(tq + COL_D + n0, r);
            tc::tmem_wait_ld();
        }
        if (is_k) {
            const float f = s_u[i] * d.out[i];
#pragma unroll
            for (int e = 0; e < NC; e += 4) {
                const float4 w = *reinterpret_cast<const float4*>(s_ds + n0 + e);
                const float us[4] = {__uint_as_float(r[e]) * (f * w.x), __uint_as_float(r[e + 1]) * (f * w.y),
                                     __uint_as_float(r[e + 2]) * (f * w.z), __uint_as_float(r[e + 3]) * (f * w.w)};
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                    const float2 y = unpack2(reinterpret_cast<const uint32_t*>(&own[e / 8])[(e + u) % 8 / 2], E());
                    kus = fmaf(y.x, us[u], fmaf(y.y, us[u + 1], kus));
                    first[e + u] += us[u];
                    first[e + u + 1] += us[u + 1];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < NC; e += 2) {
                const float2 y = unpack2(reinterpret_cast<const uint32_t*>(&own[e / 8])[e % 8 / 2], E());
                qgq = fmaf(y.x, first[e], fmaf(y.y, first[e + 1], qgq));
            }
        }
        O* dst = (is_k ? gk : gq) + go + i * gs + n0;
        if (i < n) {
#pragma unroll
            for (int e = 0; e < NC; e += 8) {
                if (n0 + e >= N) break;
                if constexpr (sizeof(O) == 2) {
                    *reinterpret_cast<uint4*>(dst + e) =
                        make_uint4(pack_as<E>(mk2(first[e], first[e + 1])), pack_as<E>(mk2(first[e + 2], first[e + 3])),
                                   pack_as<E>(mk2(first[e + 4], first[e + 5])), pack_as<E>(mk2(first[e + 6], first[e + 7])));
                } else {
                    *reinterpret_cast<float4*>(dst + e) = make_float4(first[e], first[e + 1], first[e + 2], first[e + 3]);
                    *reinterpret_cast<float4*>(dst + e + 4) = make_float4(first[e + 4], first[e + 5], first[e + 6], first[e + 7]);
                }
            }
        }
        if (is_k) {
            s_kz[part][i] = kz;
        } else {
            s_qgq[part][i] = qgq;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) kus += __shfl_xor_sync(0xffffffffu, kus, o);
        if (lane == 0) s_kus[warp] = kus;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) {
        double all = 0.0, us = 0.0;
        for (int w = 0; w < NW; ++w) {
            all += s_dot[w];
            us += (double)s_kus[w];
        }
        // <S+, dS+> = e^{G_end} <S, dS+> + sum_i e^{G_end - G_i} u_i.(dS+^T k_i)
        all = all * (double)d.all + us;
        double r[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            double qg = 0.0;
            float kzs = 0.f, gb = 0.f;
            for (int p = 0; p < NPART; ++p) {
                qg += (double)s_qgq[p][t];
                kzs += s_kz[p][t];
                gb += s_gb[p][t];
            }
            r[e] = qg - (double)d.beta[t] * (double)s_zv[t];
            if (t < n) gbeta[(t0 + t) * sh.H + h] = s_zv[t] - d.in[t] * kzs - gb;
        }
        r[0] += r[1];
        double tot = r[0];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_down_sync(0xffffffffu, tot, o);
            if (lane + o < 32) tot += up;
        }
        const double behind = tot - r[0];
        if (2 * lane < n) gg[(t0 + 2 * lane) * sh.H + h] = (float)(behind + r[0] + all);
        if (2 * lane + 1 < n) gg[(t0 + 2 * lane + 1) * sh.H + h] = (float)(behind + r[1] + all);
        if (s_gave_up) {
            if (lane == 0) {
                tc::drain_mmas(&mb_drain, kDeltaWait);
                tc::mbar_wait_bounded(&mb_ops, 0, kDeltaWait);
                if (M::LATE) tc::mbar_wait_bounded(&mb_late, 0, kDeltaWait);
                if (status) atomicOr(status, kStatusDelta);
            }
            __syncwarp();
        }
        tc::tmem_dealloc(tmem, COLS);
    }
}

Shape shape(const DeltaArgs& a) {
    const int nc = (int)((a.T + C - 1) / C);
    return Shape{(int)a.T, (int)a.H, (int)(a.H / a.KH), (int)a.N, (int)a.P, nc, 0, nc};
}
int64_t chunk_count(const DeltaArgs& a) { return a.Bz * a.H * ((a.T + C - 1) / C); }

// Workspace: the images of every chunk and value head, (the backward: those
// for its own scan too), then the operands of every chunk and key head.
size_t image_bytes(const DeltaArgs& a) { return (size_t)chunk_count(a) * Image::STRIDE; }
size_t operand_bytes(const DeltaArgs& a, bool back) {
    const uint32_t one = a.N <= 64 ? (back ? Operands<64>::BWD : Operands<64>::FWD) : back ? Operands<128>::BWD : Operands<128>::FWD;
    return (size_t)(chunk_count(a) / a.H * a.KH) * one;
}

// The prep of the shape's chunks; with `overlap` it may start while the kernel
// before it in the stream still runs.
template <typename E, int ND, bool BACK>
cudaError_t prep_tc(const DeltaArgs& a, const Shape& sh, unsigned char* image, unsigned char* image_t,
                    unsigned char* operands, bool overlap, cudaStream_t st) {
    using M = PrepSmem<ND, BACK>;
    const cudaError_t e = allow<delta_prep_tc<E, ND, BACK>>(M::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.Bz * a.H * (sh.c1 - sh.c0)));
    cfg.blockDim = dim3(PT);
    cfg.dynamicSmemBytes = M::BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, delta_prep_tc<E, ND, BACK>, static_cast<const E*>(a.q), static_cast<const E*>(a.k), a.g,
                              a.beta, a.lens, image, image_t, operands, a.scale, sh, status_word());
}

// The SMs of the current device.
cudaError_t sm_count(int* n) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
}

// The cut of n chains of nc chunks that takes the fewest chunks' time, a round
// counted as ROUND chunks more (its launch, and the state's way out and in).
Rounds cut(int64_t n, int nc, int sms, float* between) {
    constexpr int ROUND = 3;
    Rounds best{(int)n, 1, 1, 0, between};  // one launch: waves of whole chains
    double least = (double)((n + sms - 1) / sms) * nc + ROUND;
    for (int pieces = 2; n > sms && pieces <= 8 && pieces <= nc; ++pieces) {
        int rounds = (int)((n * pieces + sms - 1) / sms);
        while (pieces * ((n + rounds - 1) / rounds) > sms) ++rounds;
        const double t = rounds * ((double)((nc + pieces - 1) / pieces) + ROUND);
        if (t < least) least = t, best.pieces = pieces, best.rounds = rounds;
    }
    return best;
}
unsigned ctas(const Rounds& r) { return (unsigned)(r.pieces * ((r.n + r.rounds - 1) / r.rounds)); }
size_t state_bytes(const DeltaArgs& a) { return sizeof(float) * a.Bz * a.H * a.N * a.P; }

// Parts of a sequence that are prepared and scanned in turn, the next part's
// prep beside the scan: the scan has one CTA per head, so with fewer heads than
// SMs the prep (a CTA per chunk and head) takes the others.  One part costs two
// more launches and the state's way through memory (about 8 us), so a part has
// at least 16 chunks (40 to 60 us of scan).  In parts against whole, from a cold L2,
// 2048 tokens, 64/64: 24 heads 121 against 128 us, 48 134 and 151, 96 196 and 198
// (128/128: 272 and 280), 120 226 and 222 (318 and 316), 144 262 and 255; 16384
// tokens of 32 heads, 128/64: 1065 and 1281.
int parts_of(const DeltaArgs& a) {
    const int64_t nc = (a.T + C - 1) / C;
    if (a.Bz * a.H > 100) return 1;
    return (int)(nc < 32 ? 1 : nc / 16 < 8 ? nc / 16 : 8);
}

template <typename E, int ND>
cudaError_t forward_tc(const DeltaArgs& a, void* ws, cudaStream_t st) {
    unsigned char* image = static_cast<unsigned char*>(ws);
    unsigned char* operands = image + image_bytes(a);
    float* between = reinterpret_cast<float*>(operands + operand_bytes(a, false));  // the state from part to part
    constexpr uint32_t smem = ScanSmem<ND>::BYTES + sizeof(ScanShared);
    cudaError_t e = allow<delta_scan_tc<E, ND, false>>(smem);
    if (e == cudaSuccess) e = allow<delta_scan_tc<E, ND, true>>(smem);
    int sms = 0;
    if (e == cudaSuccess) e = sm_count(&sms);
    const int parts = parts_of(a);
    Shape sh = shape(a);
    for (int p = 0; p < parts && e == cudaSuccess; ++p) {
        sh.c0 = (int)((int64_t)sh.nc * p / parts);
        sh.c1 = (int)((int64_t)sh.nc * (p + 1) / parts);
        if ((e = prep_tc<E, ND, false>(a, sh, image, nullptr, operands, p > 0, st)) != cudaSuccess) break;
        const ScanArgs<E> g{static_cast<const E*>(a.v), image, operands, p ? between : a.h0, static_cast<E*>(a.o),
                            p + 1 < parts ? between : a.h_final, nullptr, nullptr};
        Rounds turn = cut(a.Bz * a.H, sh.c1 - sh.c0, sms, between);
        for (; turn.now < turn.rounds && e == cudaSuccess; ++turn.now) {
            if (turn.rounds > 1)
                delta_scan_tc<E, ND, true><<<ctas(turn), ST, smem, st>>>(g, a.lens, sh, turn, status_word());
            else
                delta_scan_tc<E, ND, false><<<ctas(turn), ST, smem, st>>>(g, a.lens, sh, turn, status_word());
            e = cudaGetLastError();
        }
    }
    return e;
}

template <typename E, int ND>
cudaError_t back_scans_tc(const DeltaArgs& a, void* ws, float* states, float* after, float* writes, float* zs,
                          cudaStream_t st) {
    unsigned char* image = static_cast<unsigned char*>(ws);
    unsigned char* image_t = image + image_bytes(a);
    unsigned char* operands = image_t + image_bytes(a);
    cudaError_t e = prep_tc<E, ND, true>(a, shape(a), image, image_t, operands, false, st);
    if (e != cudaSuccess) return e;
    constexpr uint32_t f = ScanSmem<ND>::BYTES + sizeof(ScanShared), r = BackSmem<ND>::BYTES + sizeof(BackShared);
    constexpr uint32_t smem = f > r ? f : r;
    if ((e = allow<delta_both_scans_tc<E, ND>>(smem)) != cudaSuccess) return e;
    const ScanArgs<E> fwd{static_cast<const E*>(a.v), image, operands, a.h0, nullptr, nullptr, states, writes};
    const BackArgs<E> back{static_cast<const E*>(a.dout), image_t, operands, a.dh_final, a.gh0, after, zs};
    int sms = 0;
    if ((e = sm_count(&sms)) != cudaSuccess) return e;
    const Shape sh = shape(a);
    Rounds turn = cut(2 * a.Bz * a.H, sh.nc, sms, reinterpret_cast<float*>(operands + operand_bytes(a, true)));
    for (; turn.now < turn.rounds && e == cudaSuccess; ++turn.now) {
        delta_both_scans_tc<E, ND><<<ctas(turn), ST, smem, st>>>(back, fwd, a.lens, sh, turn, status_word());
        e = cudaGetLastError();
    }
    return e;
}
template <typename E, typename O, int ND, int PD>
cudaError_t grad_tc(const DeltaArgs& a, const unsigned char* image_t, const unsigned char* operands, const float* states,
                    const float* after, const float* writes, const float* zs, void* gq, void* gk, cudaStream_t st) {
    using M = GradSmem<ND, PD>;
    const cudaError_t e = allow<delta_grad_tc<E, O, ND, PD>>(M::BYTES);
    if (e != cudaSuccess) return e;
    delta_grad_tc<E, O, ND, PD><<<(unsigned)chunk_count(a), M::NT, M::BYTES, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.v), static_cast<const E*>(a.dout),
        a.g, a.beta, a.lens, a.scale, image_t, operands, states, after, writes, zs, static_cast<O*>(gq),
        static_cast<O*>(gk), static_cast<E*>(a.gv), a.gg, a.gbeta, shape(a), status_word());
    return cudaGetLastError();
}
template <typename E, typename O>
cudaError_t grad_by_width(const DeltaArgs& a, void* ws, const float* states, const float* after, const float* writes,
                          const float* zs, void* gq, void* gk, cudaStream_t st) {
    const unsigned char* image_t = static_cast<const unsigned char*>(ws) + image_bytes(a);
    const unsigned char* operands = image_t + image_bytes(a);
    if (a.N <= 64)
        return a.P <= 64 ? grad_tc<E, O, 64, 64>(a, image_t, operands, states, after, writes, zs, gq, gk, st)
                         : grad_tc<E, O, 64, 128>(a, image_t, operands, states, after, writes, zs, gq, gk, st);
    return a.P <= 64 ? grad_tc<E, O, 128, 64>(a, image_t, operands, states, after, writes, zs, gq, gk, st)
                     : grad_tc<E, O, 128, 128>(a, image_t, operands, states, after, writes, zs, gq, gk, st);
}

template <typename E>
cudaError_t back_scans_by_width(const DeltaArgs& a, void* ws, float* states, float* after, float* writes, float* zs,
                                cudaStream_t st) {
    return a.N <= 64 ? back_scans_tc<E, 64>(a, ws, states, after, writes, zs, st)
                     : back_scans_tc<E, 128>(a, ws, states, after, writes, zs, st);
}

template <typename E>
cudaError_t forward_by_width(const DeltaArgs& a, void* ws, cudaStream_t st) {
    return a.N <= 64 ? forward_tc<E, 64>(a, ws, st) : forward_tc<E, 128>(a, ws, st);
}

}  // namespace

size_t tc_workspace_bytes(const DeltaArgs& a) {
    return image_bytes(a) + operand_bytes(a, false) + state_bytes(a);
}
cudaError_t launch_forward_tc(const DeltaArgs& a, void* ws, cudaStream_t st) {
    return a.dtype == CSSD_BF16 ? forward_by_width<__nv_bfloat16>(a, ws, st) : forward_by_width<__half>(a, ws, st);
}

cudaError_t launch_grad_tc(const DeltaArgs& a, void* ws, const float* states, const float* after, const float* writes,
                           const float* zs, void* gq, void* gk, cudaStream_t st) {
    const bool shared = a.H != a.KH;
    if (a.dtype == CSSD_BF16)
        return shared ? grad_by_width<__nv_bfloat16, float>(a, ws, states, after, writes, zs, gq, gk, st)
                      : grad_by_width<__nv_bfloat16, __nv_bfloat16>(a, ws, states, after, writes, zs, gq, gk, st);
    return shared ? grad_by_width<__half, float>(a, ws, states, after, writes, zs, gq, gk, st)
                  : grad_by_width<__half, __half>(a, ws, states, after, writes, zs, gq, gk, st);
}
size_t tc_back_bytes(const DeltaArgs& a) { return 2 * image_bytes(a) + operand_bytes(a, true) + 2 * state_bytes(a); }
cudaError_t launch_back_scans_tc(const DeltaArgs& a, void* ws, float* states, float* after, float* writes, float* zs,
                                 cudaStream_t st) {
    return a.dtype == CSSD_BF16 ? back_scans_by_width<__nv_bfloat16>(a, ws, states, after, writes, zs, st)
                                : back_scans_by_width<__half>(a, ws, states, after, writes, zs, st);
}

}  // namespace delta
}  // namespace cssd
