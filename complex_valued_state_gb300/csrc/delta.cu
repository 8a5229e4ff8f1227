// The gated delta rule over a sequence, in fp32 on the CUDA cores: forward and
// gradients.  Per batch row and value head, with S in R^{N x P}:
//     S' = e^{g_t} S_{t-1},  S_t = S' + k_t (beta_t (v_t - S'^T k_t))^T,
//     o_t = scale S_t^T q_t
// in chunks of 64 tokens.  With G_i the sum of g from the chunk's start, S the
// state that enters it and M_ij = e^{G_i - G_j} (i >= j), the writes
// u_i = beta_i (v_i - S'^T k_i) of a chunk solve a triangular system:
//     A_ij = beta_i M_ij k_i.k_j (i > j),  T = (I + A)^-1,  X = (M o Q K^T) T
//     R  = beta (V - e^G K S)                       64 x P
//     U  = T R,   O = scale (e^G Q S + X R)
//     S+ = e^{G_end} S + K^T (e^{G_end - G} U)
// and with W = T beta e^G K and Q' = e^G Q - X beta e^G K what a chunk asks of
// the state that enters it is two products, one behind the other:
//     [U; O] = [T; scale X] beta V + [-W; scale Q'] S
//     S+ = e^{G_end} S + K^T (e^{G_end - G} U)
// The gradients run the same chain backwards:
//     Z  = T^T (e^{G_end - G} K) dS+ + scale X^T dO        (of R)
//     dV = beta Z
//     dS = e^{G_end} dS+ - (beta e^G K)^T Z + scale (e^G Q)^T dO
// and, per chunk, with everything above at hand,
//     dQ = scale e^G dO S^T + Pm K,             Pm = scale M o (dO U^T)
//     dK = Pm^T Q + (W + W^T) K - beta e^G Z S^T + e^{G_end - G} U dS+^T,
//                                               W = -beta (M o Z U^T), i > j
//     dbeta_i = z_i.v_i - e^{G_i} k_i.(S z_i) - sum_{j<i} M_ij (k_i.k_j)(z_i.u_j)
//     dg_i = sum_{j>=i} (q_j.dq_j - v_j.dv_j) + <S+, dS+>
// (each e^{G_i} multiplies exactly what q_i reads and what v_i is compared
// with, so dL/dG_i is the difference of those two inner products).
//
// These kernels serve fp32 tensors, with plain fp32 multiply-adds from shared
// memory.  What does not wait for the state is made for all chunks at once by
// delta_prep; delta_scan and delta_both_scans walk the chunks.

#include "cssd_internal.h"
#include "delta_common.cuh"
#include "pairs.cuh"

namespace cssd {
namespace delta {
namespace {

constexpr int NT = 256;       // threads of every kernel here
constexpr int LT = C + 4;     // row stride of a 64 x 64 matrix in shared memory

struct Geo {
    int T, H, G, N, P, nc;  // G: value heads per key head
};

// rows x w elements of src (row stride `stride` elements) into dst (row
// stride ld, fp32); rows at or past n are zeros.
template <typename T>
__device__ void load_rows(float* dst, int ld, const T* src, int64_t stride, int rows, int w, int n, int tid) {
    constexpr int E = 16 / sizeof(T);
    const int per = w / E;
    for (int e = tid; e < rows * per; e += NT) {
        const int r = e / per, c = (e % per) * E;
        alignas(16) T tmp[E];
        if (r < n) {
            *reinterpret_cast<uint4*>(tmp) = *reinterpret_cast<const uint4*>(src + r * stride + c);
#pragma unroll
            for (int u = 0; u < E; ++u) dst[r * ld + c + u] = to_f(tmp[u]);
        } else {
#pragma unroll
            for (int u = 0; u < E; ++u) dst[r * ld + c + u] = 0.f;
        }
    }
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// A0 B^T and A1 B^T, rows r0 + 16 a and columns c0 + 16 c, without the 16 x 16
// blocks above the diagonal.
__device__ __forceinline__ void mm_lower_rr(float (&acc0)[4][4], float (&acc1)[4][4], const float* A0, const float* A1,
                                            int lda, const float* B, int ldb, int K, int r0, int c0) {
    for (int k = 0; k < K; k += 4) {
        float4 b[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = ld4(B + (c0 + 16 * c) * ldb + k);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const float4 u = ld4(A0 + (r0 + 16 * a) * lda + k), w = ld4(A1 + (r0 + 16 * a) * lda + k);
#pragma unroll
            for (int c = 0; c <= a; ++c) {
                acc0[a][c] = dot4(u, b[c], acc0[a][c]);
                acc1[a][c] = dot4(w, b[c], acc1[a][c]);
            }
        }
    }
}

// acc[a][c] += sum_i A[i lda + r0 + a] f[i] B[i ldb + c0 + c], i from i0 to C - 1.
__device__ __forceinline__ void mm_kr(float (&acc)[4][4], const float* A, int lda, const float* f, const float* B, int ldb,
                                      int i0, int r0, int c0) {
#pragma unroll 4
    for (int i = i0; i < C; ++i) {
        const float4 b = ld4(B + i * ldb + c0), v = ld4(A + i * lda + r0);
        const float x[4] = {v.x * f[i], v.y * f[i], v.z * f[i], v.w * f[i]};
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            acc[a][0] = fmaf(x[a], b.x, acc[a][0]);
            acc[a][1] = fmaf(x[a], b.y, acc[a][1]);
            acc[a][2] = fmaf(x[a], b.z, acc[a][2]);
            acc[a][3] = fmaf(x[a], b.w, acc[a][3]);
        }
    }
}

// t += T B and, with BOTH, x += X B for the rows r0 .. r0 + 3 of the lower
// triangular T and X (row stride LT), row j of B times f[j].
template <bool BOTH>
__device__ __forceinline__ void mm_lower(float (&t)[4][4], float (&x)[4][4], const float* T, const float* X, const float* f,
                                         const float* B, int ldb, int r0, int c0) {
    for (int k = 0; k <= r0; k += 4) {
        float4 b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            b[u] = ld4(B + (k + u) * ldb + c0);
            const float m = f[k + u];
            b[u].x *= m, b[u].y *= m, b[u].z *= m, b[u].w *= m;
        }
#pragma unroll
        for (int h = 0; h < (BOTH ? 2 : 1); ++h)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const float4 v = ld4((h ? X : T) + (r0 + a) * LT + k);
                const float w[4] = {v.x, v.y, v.z, v.w};
                float(&acc)[4] = h ? x[a] : t[a];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    acc[0] = fmaf(w[u], b[u].x, acc[0]);
                    acc[1] = fmaf(w[u], b[u].y, acc[1]);
                    acc[2] = fmaf(w[u], b[u].z, acc[2]);
                    acc[3] = fmaf(w[u], b[u].w, acc[3]);
                }
            }
    }
}
__device__ __forceinline__ void st4(float* p, const float (&v)[4], float m) {
    *reinterpret_cast<float4*>(p) = make_float4(m * v[0], m * v[1], m * v[2], m * v[3]);
}

// acc[a][c] += sum_k A[(r0 + RS a) lda + k] B[(c0 + CS c) ldb + k], K a multiple of 4.
template <int RA, int RS, int CS>
__device__ __forceinline__ void mm_rr(float (&acc)[RA][4], const float* A, int lda, const float* B, int ldb, int K,
                                      int r0, int c0) {
    for (int k = 0; k < K; k += 4) {
        float4 b[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = ld4(B + (c0 + CS * c) * ldb + k);
#pragma unroll
        for (int a = 0; a < RA; ++a) {
            const float4 v = ld4(A + (r0 + RS * a) * lda + k);
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[a][c] = dot4(v, b[c], acc[a][c]);
        }
    }
}

// --------------------------------------------------------------- what does not wait for the state
// Floats of one chunk and value head as the scans read them: the 64 rows that
// multiply the state (128 with those of the output) and the 64 rows that update
// it, all of stride N + 4, then e^{G_end}.
__host__ __device__ constexpr int image_floats(int rows, int N) { return (rows + C) * (N + 4) + 4; }

struct Made {
    float *fwd, *uo;        // forward image (128 rows; 64 for the gradients), [T; scale X] beta V (T's alone for the gradients)
    float *back, *z, *add;  // backward image, scale X^T dO [64, P], scale (e^G Q)^T dO [N, P]
};

// One CTA per chunk and value head.  Bound by shared memory, 4 x 4 outputs a
// thread reading 8 float4 for 64 multiply-adds (12 for 128 where two products
// share a factor), and by having 1.3 CTAs an SM at the sizes measured: 27 us for
// 1 x 1000 x 12, 64/64; 33 us for the gradients' 2 x 515 x 12.
template <bool BACK>
__global__ void __launch_bounds__(NT) delta_prep(const float* __restrict__ q, const float* __restrict__ k,
                                                 const float* __restrict__ v, const float* __restrict__ dout,
                                                 const float* __restrict__ g, const float* __restrict__ beta,
                                                 const int* __restrict__ lens, float scale, Made made, Geo ge) {
    extern __shared__ __align__(16) float sm[];
    __shared__ Decays d;
    __shared__ float s_bin[C], s_one[C];
    const int tid = threadIdx.x, c = blockIdx.x % ge.nc, bh = blockIdx.x / ge.nc;
    const int b = bh / ge.H, h = bh % ge.H, KH = ge.H / ge.G, N = ge.N, P = ge.P;
    const int n = min(row_len(lens, b, ge.T) - c * C, C);
    if (n <= 0) return;
    const int LK = N + 4, LP = P + 4;
    float* sk = sm;
    float* sq = sk + C * LK;
    float* sv = sq + C * LK;  // V, then dO
    float* t = sv + C * LP;
    float* x = t + C * LT;
    float* w = x + C * LT;
    const int64_t t0 = (int64_t)b * ge.T + (int64_t)c * C, ci = blockIdx.x;
    const int64_t ko = (t0 * KH + h / ge.G) * N, ks = (int64_t)KH * N, vo = (t0 * ge.H + h) * P, vs = (int64_t)ge.H * P;
    load_rows(sk, LK, k + ko, ks, C, N, n, tid);
    load_rows(sq, LK, q + ko, ks, C, N, n, tid);
    load_rows(sv, LP, v + vo, vs, C, P, n, tid);
    if (tid < 32) chunk_decays(d, g + t0 * ge.H + h, beta + t0 * ge.H + h, ge.H, n, tid);
    __syncthreads();
    if (tid < C) s_bin[tid] = d.beta[tid] * d.in[tid], s_one[tid] = 1.f;
    {
        const int ti = tid / 16, tj = tid % 16;
        float kk[4][4] = {}, qk[4][4] = {};
        mm_lower_rr(kk, qk, sk, sq, LK, sk, LK, N, ti, tj);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int i = ti + 16 * a, j = tj + 16 * y;
                const float m = i >= j ? decay_between(d, i, j) : 0.f;
                t[i * LT + j] = i > j ? d.beta[i] * (m * kk[a][y]) : 0.f;
                x[i * LT + j] = i >= j ? m * qk[a][y] : 0.f;
            }
    }
    __syncthreads();
    tri_inverse_in_place<LT>(t, w, tid);
    const int r0 = 4 * (tid / 16), c0 = 4 * (tid % 16);
    {
        float acc[4][4] = {}, none[4][4];
        mm_lower<false>(acc, none, x, nullptr, s_one, t, LT, r0, c0);
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 4; ++a) st4(x + (r0 + a) * LT + c0, acc[a], 1.f);
    }
    __syncthreads();
    float* img = made.fwd + ci * image_floats(BACK ? C : 2 * C, N);
    float* rows = img + (BACK ? C : 2 * C) * LK;  // the rows that update the state
    float* bimg = BACK ? made.back + ci * image_floats(C, N) : nullptr;
    for (int col = c0; col < N; col += 64) {
        float tk[4][4] = {}, xk[4][4] = {};
        mm_lower<!BACK>(tk, xk, t, x, s_bin, sk, LK, r0, col);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int i = r0 + a;
            const float4 kr = ld4(sk + i * LK + col);
            st4(img + i * LK + col, tk[a], -1.f);
            const float ku[4] = {kr.x, kr.y, kr.z, kr.w};
            st4(rows + i * LK + col, ku, d.out[i]);
            if constexpr (BACK) {
                st4(bimg + (C + i) * LK + col, ku, -s_bin[i]);
            } else {
                const float4 qr = ld4(sq + i * LK + col);
                const float in = d.in[i];
                const float y[4] = {fmaf(in, qr.x, -xk[a][0]), fmaf(in, qr.y, -xk[a][1]), fmaf(in, qr.z, -xk[a][2]),
                                    fmaf(in, qr.w, -xk[a][3])};
                st4(img + (C + i) * LK + col, y, scale);
            }
        }
        if constexpr (BACK) {
            float wk[4][4] = {};
            mm_kr(wk, t, LT, d.out, sk, LK, r0, r0, col);
#pragma unroll
            for (int a = 0; a < 4; ++a) st4(bimg + (r0 + a) * LK + col, wk[a], 1.f);
        }
    }
    if (tid < 4) {
        rows[C * LK + tid] = d.all;
        if (BACK) bimg[2 * C * LK + tid] = d.all;
    }
    float* uo = made.uo + ci * (BACK ? C : 2 * C) * P;
    for (int col = c0; col < P; col += 64) {
        float tv[4][4] = {}, xv[4][4] = {};
        mm_lower<!BACK>(tv, xv, t, x, d.beta, sv, LP, r0, col);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            st4(uo + (r0 + a) * P + col, tv[a], 1.f);
            if (!BACK) st4(uo + (C + r0 + a) * P + col, xv[a], scale);
        }
    }
    if constexpr (BACK) {
        __syncthreads();
        load_rows(sv, LP, dout + vo, vs, C, P, n, tid);
        __syncthreads();
        float* z = made.z + ci * C * P;
        float* add = made.add + ci * N * P;
        for (int col = c0; col < P; col += 64) {
            float xd[4][4] = {};
            mm_kr(xd, x, LT, s_one, sv, LP, r0, r0, col);
#pragma unroll
            for (int a = 0; a < 4; ++a) st4(z + (r0 + a) * P + col, xd[a], scale);
            for (int r = r0; r < N; r += 64) {
                float qd[4][4] = {};
                mm_kr(qd, sq, LK, d.in, sv, LP, 0, r, col);
#pragma unroll
                for (int a = 0; a < 4; ++a) st4(add + (r + a) * P + col, qd[a], scale);
            }
        }
    }
}

// --------------------------------------------------------------- the scans
// One CTA per value head and slice of PW state columns (they never mix),
// walking the chunks with the next chunk's image on its way (cp.async).  Shared
// memory hands a warp 128 bytes a cycle, the same word to all lanes or not, so
// what bounds both products is the bytes a thread reads for a multiply-add:
// tiles of 4 rows x 4 columns (2 bytes; a row x 8 columns, 4.5, took twice as
// long), the sum split over neighbouring lanes so that every thread has a tile
// and joined by shuffles, which leave each lane its rows of the tile.
struct ScanIo {
    const float *img, *init, *add;  // as made; add: forward null
    const float* s0;                // the state before the first chunk, or null
    float* s_end;                   // after the last, or null
    float* kept;                    // the state entering each chunk (backward: leaving), or null
    float* made;                    // the first 64 rows of the first product, U or Z, or null
    float* o;                       // outputs (ROWS = 128)
};

// Up to this many CTAs of 16 columns, half of the SMs, a CTA takes 8 with half
// the threads.  1000 tokens from a cold L2, 64/64: 48 CTAs 71 us against 79, 76 72
// against 79, 96 108 against 106, 152 116 against 110; 128/128: 48 93 against 119,
// 96 179 against 152.
constexpr int NARROW = 76;
constexpr int scan_threads(int PW) { return 16 * PW; }
__host__ __device__ constexpr int state_stride(int rows, int N) { return (N + 31) / 32 * 32 + 4 * (256 / rows); }

template <int ROWS, int PW>
constexpr uint32_t scan_smem(int N) {
    return sizeof(float) * (2 * image_floats(ROWS, N) + PW * state_stride(ROWS, N) + C * (PW + 8));
}

template <int ROWS, int ND, int PW, bool BACK>
__device__ __forceinline__ void scan_body(const ScanIo& io, int bh, int p0, const int* __restrict__ lens, const Geo& ge,
                                          float* sm) {
    // Lanes that share a tile of the first product (ROWS x PW) and of the second
    // (ND x PW), and the rows each is left with.
    constexpr int S1 = 256 / ROWS, S2 = 256 / ND, R1 = 4 / S1, R2 = 4 / S2;
    constexpr int NT = scan_threads(PW), X = PW / 4, LU = PW + 8;  // tiles across, row stride of U
    const int tid = threadIdx.x, b = bh / ge.H, h = bh % ge.H, N = ge.N, P = ge.P, LA = N + 4;
    const int LS = state_stride(ROWS, N);
    const int len = row_len(lens, b, ge.T), nck = (len + C - 1) / C;
    const int image = image_floats(ROWS, N);
    float* st = sm + 2 * image;  // the state: column 4 x + i of the slice in row X i + x
    float* su = st + PW * LS;    // U or Z, [64][LU]
    const int l1 = tid % S1, x1 = tid / S1 % X, tile1 = tid / (X * S1) * 4, row = tile1 + R1 * l1;
    const int l2 = tid % S2, x2 = tid / S2 % X, tile2 = tid / (X * S2) * 4, nr = tile2 + R2 * l2;
    // Whether this thread's rows of the state are there, the same for the S2 lanes of
    // a tile, and whether any of its warp's are: a warp has 16 rows, or 32 (ND = 128
    // in slices of 8 columns), and N, a multiple of 16, may end inside those.  What
    // shuffles goes by the warp.
    const bool there = tile2 < N, warp_there = (tid & ~31) / (X * S2) * 4 < N;
    const int64_t so = ((int64_t)bh * N + nr) * P + p0 + 4 * x2;  // this thread's state
    auto load = [&](int c, int buf) {
        const float* src = io.img + ((int64_t)bh * ge.nc + c) * image;
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(sm + buf * image);
        for (int e = tid; e < image / 4; e += NT)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * e), "l"(src + 4 * e) : "memory");
    };
    float4 init[R1], add[R2];
    auto load_init = [&](int c) {
        const float* src = io.init + (((int64_t)bh * ge.nc + c) * ROWS + row) * P + p0 + 4 * x1;
#pragma unroll
        for (int a = 0; a < R1; ++a) init[a] = ld4(src + a * P);
        if (BACK && there) {
            const float* more = io.add + (((int64_t)bh * ge.nc + c) * N + nr) * P + p0 + 4 * x2;
#pragma unroll
            for (int a = 0; a < R2; ++a) add[a] = ld4(more + a * P);
        }
    };
    float s[R2][4];
#pragma unroll
    for (int a = 0; a < R2; ++a) {
        const float4 v = io.s0 && there ? ld4(io.s0 + so + a * P) : make_float4(0.f, 0.f, 0.f, 0.f);
        s[a][0] = v.x, s[a][1] = v.y, s[a][2] = v.z, s[a][3] = v.w;
    }
    auto put_state = [&] {
#pragma unroll
        for (int a = 0; a < R2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) st[(X * i + x2) * LS + nr + a] = s[a][i];
    };
    auto chunk = [&](int it) { return BACK ? nck - 1 - it : it; };
    if (there) put_state();
    if (nck > 0) {
        load(chunk(0), 0);
        load_init(chunk(0));
    }
    for (int it = 0; it < nck; ++it) {
        const int c = chunk(it);
        const int64_t ci = (int64_t)bh * ge.nc + c;
        const float* img = sm + (it & 1) * image;
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (it + 1 < nck) load(chunk(it + 1), (it + 1) & 1);
        {
            f2 acc[4][4] = {};  // sums over even and odd k
#pragma unroll 2
            for (int e = 4 * l1; e < N; e += 4 * S1) {
                ulonglong2 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(st + (X * i + x1) * LS + e);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(img + (tile1 + a) * LA + e);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][i] = fma2(w.y, x[i].y, fma2(w.x, x[i].x, acc[a][i]));
                }
            }
            float y[4][4];
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[a][i] = sum2(acc[a][i]);
            join<S1>(y, l1);
#pragma unroll
            for (int a = 0; a < R1; ++a) {
                const float4 z = make_float4(y[a][0] + init[a].x, y[a][1] + init[a].y, y[a][2] + init[a].z, y[a][3] + init[a].w);
                const int r = row + a;
                if (ROWS == C || tile1 < C) {
                    *reinterpret_cast<float4*>(su + r * LU + 4 * x1) = z;
                    if (io.made) *reinterpret_cast<float4*>(io.made + (ci * C + r) * P + p0 + 4 * x1) = z;
                } else if (c * C + r - C < len) {
                    *reinterpret_cast<float4*>(io.o + (((int64_t)b * ge.T + (int64_t)c * C + r - C) * ge.H + h) * P + p0 + 4 * x1) = z;
                }
            }
        }
        float4 more[R2];
        if (BACK)
#pragma unroll
            for (int a = 0; a < R2; ++a) more[a] = add[a];
        if (it + 1 < nck) load_init(chunk(it + 1));
        __syncthreads();
        if (warp_there) {
            const float* ku = img + ROWS * LA + min(tile2, N - 4);  // (lanes without rows: any that are there)
            f2 d[2][4] = {};  // pairs of rows
#pragma unroll 4
            for (int i = l2; i < C; i += S2) {
                const ulonglong2 kv = *reinterpret_cast<const ulonglong2*>(ku + i * LA);
                const float4 u = ld4(su + i * LU + 4 * x2);
                const float w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const f2 u2 = mk2(w[y], w[y]);
                    d[0][y] = fma2(kv.x, u2, d[0][y]);
                    d[1][y] = fma2(kv.y, u2, d[1][y]);
                }
            }
            float y[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) un2(d[0][i], y[0][i], y[1][i]), un2(d[1][i], y[2][i], y[3][i]);
            join<S2>(y, l2);
            if (there) {
                if (io.kept)
#pragma unroll
                    for (int a = 0; a < R2; ++a)
                        *reinterpret_cast<float4*>(io.kept + (ci * N + nr + a) * P + p0 + 4 * x2) =
                            make_float4(s[a][0], s[a][1], s[a][2], s[a][3]);
                const float all = img[(ROWS + C) * LA];
#pragma unroll
                for (int a = 0; a < R2; ++a) {
                    if (BACK) y[a][0] += more[a].x, y[a][1] += more[a].y, y[a][2] += more[a].z, y[a][3] += more[a].w;
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[a][i] = fmaf(all, s[a][i], y[a][i]);
                }
                put_state();
            }
        }
    }
    if (io.s_end && there)
#pragma unroll
        for (int a = 0; a < R2; ++a)
            *reinterpret_cast<float4*>(io.s_end + so + a * P) = make_float4(s[a][0], s[a][1], s[a][2], s[a][3]);
    if (ROWS > C)  // behind the row's last token
        for (int64_t e = tid; e < (int64_t)(ge.T - len) * PW; e += NT)
            io.o[(((int64_t)b * ge.T + len + e / PW) * ge.H + h) * P + p0 + e % PW] = 0.f;
}

template <int ND, int PW>
__global__ void __launch_bounds__(scan_threads(PW)) delta_scan(ScanIo io, const int* __restrict__ lens, Geo ge) {
    extern __shared__ __align__(16) float sm[];
    const int np = ge.P / PW;
    scan_body<2 * C, ND, PW, false>(io, blockIdx.x / np, (int)(blockIdx.x % np) * PW, lens, ge, sm);
}

// Both of the gradients' scans, which do not need one another (2 x 515 x 12,
// 64/64: 37 us; one behind the other, with three products a chunk, they took 199).
template <int ND>
__global__ void __launch_bounds__(scan_threads(16)) delta_both_scans(ScanIo back, ScanIo fwd, const int* __restrict__ lens, Geo ge) {
    extern __shared__ __align__(16) float sm[];
    constexpr int PW = 16;
    const int np = ge.P / PW, half = gridDim.x / 2, i = blockIdx.x % half;
    if ((int)blockIdx.x < half)
        scan_body<C, ND, PW, true>(back, i / np, i % np * PW, lens, ge, sm);
    else
        scan_body<C, ND, PW, false>(fwd, i / np, i % np * PW, lens, ge, sm);
}

// --------------------------------------------------------------- dQ, dK, dV, dg, dbeta
// One CTA per chunk and value head.  gq and gk are the key heads' gradients
// when every value head has its own key head, else this value head's part in
// fp32, summed over the group by delta_sum_heads in a fixed order.  Bound by
// shared memory (2.3 bytes a multiply-add) at two CTAs an SM: 2 x 515 x 12, 64/64
// 61 us; with a matrix each for Pm and W, one CTA an SM, 84.
template <typename E, typename O>
__global__ void __launch_bounds__(NT) delta_grad(const E* __restrict__ q, const E* __restrict__ k,
                                                 const E* __restrict__ v, const float* __restrict__ g,
                                                 const float* __restrict__ beta, const E* __restrict__ dout,
                                                 const int* __restrict__ lens, float scale,
                                                 const float* __restrict__ states, const float* __restrict__ after,
                                                 const float* __restrict__ writes, const float* __restrict__ zs,
                                                 O* __restrict__ gq, O* __restrict__ gk, E* __restrict__ gv,
                                                 float* __restrict__ gg,
                                                 float* __restrict__ gbeta, Geo ge) {
    extern __shared__ __align__(16) float sm[];
    __shared__ Decays d;
    __shared__ float s_qgq[C], s_kz[C], s_zv[C], s_gb[C];
    __shared__ double s_dot[NT / 32];
    const int tid = threadIdx.x, c = blockIdx.x % ge.nc, bh = blockIdx.x / ge.nc;
    const int b = bh / ge.H, h = bh % ge.H, KH = ge.H / ge.G, N = ge.N, P = ge.P;
    const int len = row_len(lens, b, ge.T), n = min(len - c * C, C), here = min(ge.T - c * C, C);
    const int64_t t0 = (int64_t)b * ge.T + (int64_t)c * C, ci = (int64_t)bh * ge.nc + c;
    const int64_t ko = (t0 * KH + h / ge.G) * N, ks = (int64_t)KH * N, vo = (t0 * ge.H + h) * P, vs = (int64_t)ge.H * P;
    const int64_t go = (t0 * ge.H + h) * N, gs = (int64_t)ge.H * N;  // of gq and gk: the same as ko when G = 1
    if (n < here) {  // tokens that are not there
        const int from = max(n, 0);
        for (int e = tid; e < (here - from) * N; e += NT) {
            gq[go + (from + e / N) * gs + e % N] = from_f<O>(0.f);
            gk[go + (from + e / N) * gs + e % N] = from_f<O>(0.f);
        }
        for (int e = tid; e < (here - from) * P; e += NT) gv[vo + (from + e / P) * vs + e % P] = from_f<E>(0.f);
        for (int i = from + tid; i < here; i += NT) gg[(t0 + i) * ge.H + h] = gbeta[(t0 + i) * ge.H + h] = 0.f;
    }
    if (n <= 0) return;
    const int LK = N + 4, LP = P + 4;
    float* so = sm;  // dO
    float* sz = so + C * LP;
    float* su = sz + C * LP;
    float* sk = su + C * LP;
    float* sq = sk + C * LK;
    float* pw = sq + C * LK;  // Pm and, above the diagonal, W^T
    float* sb = pw + C * LT;  // 32 rows of S, then of dS+
    load_rows(so, LP, dout + vo, vs, C, P, n, tid);
    load_rows(sz, LP, zs + ci * C * P, P, C, P, C, tid);
    load_rows(su, LP, writes + ci * C * P, P, C, P, C, tid);
    load_rows(sk, LK, k + ko, ks, C, N, n, tid);
    load_rows(sq, LK, q + ko, ks, C, N, n, tid);
    if (tid < 32) chunk_decays(d, g + t0 * ge.H + h, beta + t0 * ge.H + h, ge.H, n, tid);
    __syncthreads();
    for (int e = tid; e < n * P; e += NT) gv[vo + (e / P) * vs + e % P] = from_f<E>(d.beta[e / P] * sz[(e / P) * LP + e % P]);
    {
        const int i = tid / 4, l = tid % 4;  // z.v
        float zv = 0.f;
        if (i < n)
            for (int p = l; p < P; p += 4) zv = fmaf(sz[i * LP + p], to_f(v[vo + i * vs + p]), zv);
        zv += __shfl_xor_sync(0xffffffffu, zv, 1);
        zv += __shfl_xor_sync(0xffffffffu, zv, 2);
        if (l == 0) s_zv[i] = zv;
    }
    {
        const int ti = tid / 16, tj = tid % 16;
        float du[4][4] = {}, zu[4][4] = {}, kk[4][4] = {};
        mm_lower_rr(du, zu, so, sz, LP, su, LP, P, ti, tj);
        mm_rr<4, 16, 16>(kk, sk, LK, sk, LK, N, ti, tj);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int i = ti + 16 * x;
            float gb = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int j = tj + 16 * y;
                const float m = i >= j ? decay_between(d, i, j) : 0.f;
                if (i >= j) pw[i * LT + j] = scale * (m * du[x][y]);
                if (i > j) {
                    const float z = m * zu[x][y];
                    gb = fmaf(z, kk[x][y], gb);
                    pw[j * LT + i] = -d.beta[i] * z;
                }
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) gb += __shfl_xor_sync(0xffffffffu, gb, o);
            if (tj == 0) s_gb[i] = gb;
        }
    }
    const int rg = tid / 8, cg = tid % 8;
    float qgq[2] = {}, kz[2] = {}, kus = 0.f;
    double dot = 0.0;
    for (int nb = 0; nb < N; nb += 32) {
        const int rows = min(32, N - nb);
        __syncthreads();
        load_rows(sb, LP, states + ci * N * P + (int64_t)nb * P, P, 32, P, rows, tid);
        __syncthreads();
        float aq[2][4] = {}, az[2][4] = {}, au[2][4] = {};
        for (int e = 0; e < P; e += 4) {
            float4 x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) x[y] = ld4(sb + (cg + 8 * y) * LP + e);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const float4 u = ld4(so + (rg + 32 * a) * LP + e), w = ld4(sz + (rg + 32 * a) * LP + e);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    aq[a][y] = dot4(u, x[y], aq[a][y]);
                    az[a][y] = dot4(w, x[y], az[a][y]);
                }
            }
        }
        __syncthreads();
        float part = 0.f;
        for (int e = tid; e < rows * P; e += NT) {
            const int r = e / P, p = e % P;
            const float x = after[ci * N * P + (int64_t)(nb + r) * P + p];
            part = fmaf(sb[r * LP + p], x, part);
            sb[r * LP + p] = x;
        }
        dot += (double)part;
        __syncthreads();
        mm_rr<2, 32, 8>(au, su, LP, sb, LP, P, rg, cg);
        float qv[2][4], kv[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int i = rg + 32 * x;
                qv[x][y] = scale * d.in[i] * aq[x][y];
                kv[x][y] = d.out[i] * au[x][y] - d.beta[i] * d.in[i] * az[x][y];
            }
        // rows j by fours: before a warp's four rows i only Pm_ij and W_ij, behind
        // them only Pm_ji and W_ji (columns past N read a padding or another row
        // that is there; they are not kept)
        for (int j = 0; j < C; j += 4) {
            float kr[4][4], qr[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int col = min(nb + cg + 8 * y, N - 1);
                    kr[u][y] = sk[(j + u) * LK + col], qr[u][y] = sq[(j + u) * LK + col];
                }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = rg + 32 * x, first = rg / 4 * 4 + 32 * x;
                const float4 r = ld4(pw + i * LT + j);
                const float a[4] = {r.x, r.y, r.z, r.w};  // (i, j), and (j, i):
                const float t[4] = {pw[j * LT + i], pw[(j + 1) * LT + i], pw[(j + 2) * LT + i], pw[(j + 3) * LT + i]};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (j < first) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            qv[x][y] = fmaf(a[u], kr[u][y], qv[x][y]);
                            kv[x][y] = fmaf(t[u], kr[u][y], kv[x][y]);
                        }
                    } else if (j > first) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) kv[x][y] = fmaf(t[u], qr[u][y], fmaf(a[u], kr[u][y], kv[x][y]));
                    } else {
                        const int k = j + u;
                        const float p1 = k <= i ? a[u] : 0.f, p2 = k >= i ? t[u] : 0.f, p3 = k < i ? t[u] : k > i ? a[u] : 0.f;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            qv[x][y] = fmaf(p1, kr[u][y], qv[x][y]);
                            kv[x][y] = fmaf(p2, qr[u][y], fmaf(p3, kr[u][y], kv[x][y]));
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = rg + 32 * x;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int col = nb + cg + 8 * y;
                if (col >= N) continue;
                qgq[x] = fmaf(sq[i * LK + col], qv[x][y], qgq[x]);
                kz[x] = fmaf(sk[i * LK + col], az[x][y], kz[x]);
                kus = fmaf(d.out[i] * sk[i * LK + col], au[x][y], kus);
                if (i < n) {
                    gq[go + i * gs + col] = from_f<O>(qv[x][y]);
                    gk[go + i * gs + col] = from_f<O>(kv[x][y]);
                }
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            qgq[x] += __shfl_xor_sync(0xffffffffu, qgq[x], o);
            kz[x] += __shfl_xor_sync(0xffffffffu, kz[x], o);
        }
        if (cg == 0) {
            s_qgq[rg + 32 * x] = qgq[x];
            s_kz[rg + 32 * x] = kz[x];
        }
    }
    dot = dot * (double)d.all + (double)kus;  // <S+, dS+> = e^{G_end} <S, dS+> + sum_i e^{G_end - G_i} u_i.(dS+^T k_i)
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (tid % 32 == 0) s_dot[tid / 32] = dot;
    __syncthreads();
    if (tid < 32) {
        double all = 0.0;
        for (int w = 0; w < NT / 32; ++w) all += s_dot[w];
        double r[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * tid + e;
            r[e] = (double)s_qgq[i] - (double)d.beta[i] * (double)s_zv[i];
            if (i < n) gbeta[(t0 + i) * ge.H + h] = s_zv[i] - d.in[i] * s_kz[i] - s_gb[i];
        }
        r[0] += r[1];
        double tot = r[0];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_down_sync(0xffffffffu, tot, o);
            if (tid + o < 32) tot += up;
        }
        const double behind = tot - r[0];
        if (2 * tid < n) gg[(t0 + 2 * tid) * ge.H + h] = (float)(behind + r[0] + all);
        if (2 * tid + 1 < n) gg[(t0 + 2 * tid + 1) * ge.H + h] = (float)(behind + r[1] + all);
    }
}

// [rows, KH, G, N] fp32 -> [rows, KH, N], summed over G in order; of two
// arrays, by blockIdx.y.
template <typename E>
__global__ void __launch_bounds__(256) delta_sum_heads(const float4* __restrict__ part0, const float4* __restrict__ part1,
                                                       E* __restrict__ out0, E* __restrict__ out1, int64_t n4, int G,
                                                       int N4) {
    const float4* part = blockIdx.y ? part1 : part0;
    E* out = blockIdx.y ? out1 : out0;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n4; e += (int64_t)gridDim.x * 256) {
        const float4* p = part + (e / N4) * G * N4 + e % N4;
        float4 s = p[0];
        for (int i = 1; i < G; ++i) {
            const float4 x = p[(int64_t)i * N4];
            s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
        }
        E* o = out + 4 * e;
        o[0] = from_f<E>(s.x), o[1] = from_f<E>(s.y), o[2] = from_f<E>(s.z), o[3] = from_f<E>(s.w);
    }
}

int64_t chunks(const DeltaArgs& a) { return (a.T + C - 1) / C; }
size_t state_floats(const DeltaArgs& a) { return (size_t)(a.Bz * a.H * chunks(a)) * a.N * a.P; }
size_t write_floats(const DeltaArgs& a) { return (size_t)(a.Bz * a.H * chunks(a)) * C * a.P; }
size_t part_floats(const DeltaArgs& a) { return a.H == a.KH ? 0 : (size_t)(a.Bz * a.T * a.H) * a.N; }

Geo geo(const DeltaArgs& a) {
    return Geo{(int)a.T, (int)a.H, (int)(a.H / a.KH), (int)a.N, (int)a.P, (int)chunks(a)};
}
// What delta_prep makes, laid out in the workspace.
Made made_in(const DeltaArgs& a, float* ws, bool back) {
    const int64_t n = a.Bz * a.H * chunks(a);
    Made m{};
    m.fwd = ws;
    m.uo = m.fwd + n * image_floats(back ? C : 2 * C, (int)a.N);
    m.back = m.uo + n * (back ? C : 2 * C) * a.P;
    m.z = m.back + (back ? n * image_floats(C, (int)a.N) : 0);
    m.add = m.z + (back ? n * C * a.P : 0);
    return m;
}
size_t made_floats(const DeltaArgs& a, bool back) {
    const int64_t n = a.Bz * a.H * chunks(a);
    const int64_t one = image_floats(back ? C : 2 * C, (int)a.N) + (back ? C : 2 * C) * a.P;
    return (size_t)(n * (one + (back ? image_floats(C, (int)a.N) + (C + a.N) * a.P : 0)));
}

template <bool BACK>
cudaError_t prep(const DeltaArgs& a, const Made& m, cudaStream_t st) {
    auto bytes = [](int64_t N, int64_t P) {
        return (uint32_t)(sizeof(float) * (2 * C * (N + 4) + C * (P + 4) + 2 * C * LT + kInverseScratch));
    };
    const uint32_t sm = bytes(a.N, a.P);
    const cudaError_t e = allow<delta_prep<BACK>>(bytes(128, 128));
    if (e != cudaSuccess) return e;
    delta_prep<BACK><<<(unsigned)(a.Bz * a.H * chunks(a)), NT, sm, st>>>(
        static_cast<const float*>(a.q), static_cast<const float*>(a.k), static_cast<const float*>(a.v),
        static_cast<const float*>(a.dout), a.g, a.beta, a.lens, a.scale, m, geo(a));
    return cudaGetLastError();
}

template <int ND, int PW>
cudaError_t scan(const DeltaArgs& a, const ScanIo& io, cudaStream_t st) {
    const uint32_t sm = scan_smem<2 * C, PW>((int)a.N);
    const cudaError_t e = allow<delta_scan<ND, PW>>(scan_smem<2 * C, PW>(ND));
    if (e != cudaSuccess) return e;
    delta_scan<ND, PW><<<(unsigned)(a.Bz * a.H * (a.P / PW)), scan_threads(PW), sm, st>>>(io, a.lens, geo(a));
    return cudaGetLastError();
}
template <int ND>
cudaError_t scan_by_heads(const DeltaArgs& a, const ScanIo& io, cudaStream_t st) {
    return a.Bz * a.H * (a.P / 16) <= NARROW ? scan<ND, 8>(a, io, st) : scan<ND, 16>(a, io, st);
}
template <int ND>
cudaError_t both(const DeltaArgs& a, const ScanIo& back, const ScanIo& fwd, cudaStream_t st) {
    const uint32_t sm = scan_smem<C, 16>((int)a.N);
    const cudaError_t e = allow<delta_both_scans<ND>>(scan_smem<C, 16>(ND));
    if (e != cudaSuccess) return e;
    delta_both_scans<ND><<<(unsigned)(2 * a.Bz * a.H * (a.P / 16)), scan_threads(16), sm, st>>>(back, fwd, a.lens, geo(a));
    return cudaGetLastError();
}

cudaError_t forward(const DeltaArgs& a, void* ws, cudaStream_t st) {
    const Made m = made_in(a, static_cast<float*>(ws), false);
    const cudaError_t e = prep<false>(a, m, st);
    if (e != cudaSuccess) return e;
    const ScanIo io{m.fwd, m.uo, nullptr, a.h0, a.h_final, nullptr, nullptr, static_cast<float*>(a.o)};
    return a.N <= 64 ? scan_by_heads<64>(a, io, st) : scan_by_heads<128>(a, io, st);
}
cudaError_t both_scans(const DeltaArgs& a, float* ws, float* states, float* after, float* writes, float* zs,
                       cudaStream_t st) {
    const Made m = made_in(a, ws, true);
    const cudaError_t e = prep<true>(a, m, st);
    if (e != cudaSuccess) return e;
    const ScanIo fwd{m.fwd, m.uo, nullptr, a.h0, nullptr, states, writes, nullptr};
    const ScanIo back{m.back, m.z, m.add, a.dh_final, a.gh0, after, zs, nullptr};
    return a.N <= 64 ? both<64>(a, back, fwd, st) : both<128>(a, back, fwd, st);
}

template <typename E, typename O>
cudaError_t grad(const DeltaArgs& a, const float* states, const float* after, const float* writes, const float* zs,
                 void* gq, void* gk, cudaStream_t st) {
    auto bytes = [](int64_t N, int64_t P) {
        return (uint32_t)(sizeof(float) * (3 * C * (P + 4) + 2 * C * (N + 4) + C * LT + 32 * (P + 4)));
    };
    const uint32_t sm = bytes(a.N, a.P);
    cudaError_t e = allow<delta_grad<E, O>>(bytes(128, 128));
    if (e != cudaSuccess) return e;
    delta_grad<E, O><<<(unsigned)(a.Bz * a.H * chunks(a)), NT, sm, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.v), a.g, a.beta,
        static_cast<const E*>(a.dout), a.lens, a.scale, states, after, writes, zs, static_cast<O*>(gq),
        static_cast<O*>(gk), static_cast<E*>(a.gv), a.gg, a.gbeta, geo(a));
    return cudaGetLastError();
}

template <typename E>
cudaError_t backward(const DeltaArgs& a, void* ws, cudaStream_t st) {
    constexpr bool TC = sizeof(E) == 2;  // 16-bit types: the tensor-core kernels
    float* states = static_cast<float*>(ws);
    float* after = states + state_floats(a);
    float* writes = after + state_floats(a);
    float* zs = writes + write_floats(a);
    float* pq = zs + write_floats(a);
    float* pk = pq + part_floats(a);
    float* rest = pk + part_floats(a);  // what prep makes; the tensor-core kernels' own
    cudaError_t e;
    if constexpr (TC) {
        e = launch_back_scans_tc(a, rest, states, after, writes, zs, st);
    } else {
        e = both_scans(a, rest, states, after, writes, zs, st);
    }
    if (e != cudaSuccess) return e;
    // key heads that are shared: a part per value head, summed in order
    const bool shared = a.H != a.KH;
    if constexpr (TC)
        e = launch_grad_tc(a, rest, states, after, writes, zs, shared ? pq : a.gq, shared ? pk : a.gk, st);
    else
        e = grad<E, float>(a, states, after, writes, zs, shared ? pq : a.gq, shared ? pk : a.gk, st);
    if (e != cudaSuccess || !shared) return e;
    const int64_t n4 = a.Bz * a.T * a.KH * (a.N / 4);
    const unsigned grid = (unsigned)((n4 + 255) / 256 < 65535 ? (n4 + 255) / 256 : 65535);
    delta_sum_heads<E><<<dim3(grid, 2), 256, 0, st>>>(reinterpret_cast<const float4*>(pq), reinterpret_cast<const float4*>(pk),
                                                      static_cast<E*>(a.gq), static_cast<E*>(a.gk), n4,
                                                      (int)(a.H / a.KH), (int)(a.N / 4));
    return cudaGetLastError();
}

}  // namespace
}  // namespace delta

size_t delta_workspace_bytes(const DeltaArgs& a) {
    return a.dtype == CSSD_F32 ? sizeof(float) * delta::made_floats(a, false) : delta::tc_workspace_bytes(a);
}
size_t delta_backward_workspace_bytes(const DeltaArgs& a) {
    return sizeof(float) * (2 * delta::state_floats(a) + 2 * delta::write_floats(a) + 2 * delta::part_floats(a)) +
           (a.dtype == CSSD_F32 ? sizeof(float) * delta::made_floats(a, true) : delta::tc_back_bytes(a));
}

cudaError_t launch_delta_forward(const DeltaArgs& a, void* ws, cudaStream_t st) {
    return a.dtype == CSSD_F32 ? delta::forward(a, ws, st) : delta::launch_forward_tc(a, ws, st);
}
cudaError_t launch_delta_backward(const DeltaArgs& a, void* ws, cudaStream_t st) {
    if (a.dtype == CSSD_BF16) return delta::backward<__nv_bfloat16>(a, ws, st);
    if (a.dtype == CSSD_F16) return delta::backward<__half>(a, ws, st);
    return delta::backward<float>(a, ws, st);
}

}  // namespace cssd
