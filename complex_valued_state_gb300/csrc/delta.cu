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
// so that T and X are made for all chunks at once and only three products a
// chunk wait for the state.  The gradients run the same chain backwards:
//     Z  = T^T (e^{G_end - G} K dS+) + scale X^T dO        (of R)
//     dV = beta Z
//     dS = e^{G_end} dS+ + scale (e^G Q)^T dO - (e^G K)^T (beta Z)
// and, per chunk, with everything above at hand,
//     dQ = scale e^G dO S^T + Pm K,             Pm = scale M o (dO U^T)
//     dK = Pm^T Q + (W + W^T) K - beta e^G Z S^T + e^{G_end - G} U dS+^T,
//                                               W = -beta (M o Z U^T), i > j
//     dbeta_i = z_i.v_i - e^{G_i} k_i.(S z_i) - sum_{j<i} M_ij (k_i.k_j)(z_i.u_j)
//     dg_i = sum_{j>=i} (q_j.dq_j - v_j.dv_j) + <S+, dS+>
// (each e^{G_i} multiplies exactly what q_i reads and what v_i is compared
// with, so dL/dG_i is the difference of those two inner products).
//
// These kernels serve fp32 tensors (and hold the sums, the states and every
// intermediate of the 16-bit ones too where those take them): the products
// are plain fp32 multiply-adds from shared memory, 4 x 4 outputs a thread.

#include "cssd_internal.h"
#include "delta_common.cuh"

namespace cssd {
namespace delta {
namespace {

constexpr int NT = 256;       // threads of every kernel here
constexpr int LT = C + 4;     // row stride of a 64 x 64 matrix in shared memory
constexpr int PW = 32;        // state columns a scan CTA owns
constexpr int LS = PW + 4;    // their row stride

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

// rows x PW columns from column p0 of an array with `width` columns (zeros
// past it and past row n).
template <typename T>
__device__ void load_slice(float* dst, const T* src, int64_t stride, int rows, int p0, int width, int n, int tid) {
    for (int e = tid; e < rows * PW; e += NT) {
        const int r = e / PW, c = e % PW;
        dst[r * LS + c] = (r < n && p0 + c < width) ? to_f(src[r * stride + p0 + c]) : 0.f;
    }
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// acc[a][c] += sum_k A[(r0 + RS a) lda + k] B[k ldb + c0 + c], K a multiple of 4.
template <int RA, int RS>
__device__ __forceinline__ void mm_rk(float (&acc)[RA][4], const float* A, int lda, const float* B, int ldb, int K,
                                      int r0, int c0) {
    for (int k = 0; k < K; k += 4) {
        float4 b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) b[u] = ld4(B + (k + u) * ldb + c0);
#pragma unroll
        for (int a = 0; a < RA; ++a) {
            const float4 v = ld4(A + (r0 + RS * a) * lda + k);
            const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                acc[a][0] = fmaf(w[u], b[u].x, acc[a][0]);
                acc[a][1] = fmaf(w[u], b[u].y, acc[a][1]);
                acc[a][2] = fmaf(w[u], b[u].z, acc[a][2]);
                acc[a][3] = fmaf(w[u], b[u].w, acc[a][3]);
            }
        }
    }
}

// acc[a][c] += sum_i A[i lda + r0 + a] B[i ldb + c0 + c].
template <int RA>
__device__ __forceinline__ void mm_kr(float (&acc)[RA][4], const float* A, int lda, const float* B, int ldb, int K,
                                      int r0, int c0) {
#pragma unroll 4
    for (int i = 0; i < K; ++i) {
        const float4 b = ld4(B + i * ldb + c0);
#pragma unroll
        for (int a = 0; a < RA; ++a) {
            const float v = A[i * lda + r0 + a];
            acc[a][0] = fmaf(v, b.x, acc[a][0]);
            acc[a][1] = fmaf(v, b.y, acc[a][1]);
            acc[a][2] = fmaf(v, b.z, acc[a][2]);
            acc[a][3] = fmaf(v, b.w, acc[a][3]);
        }
    }
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
            for (int c = 0; c < 4; ++c)
                acc[a][c] = fmaf(v.x, b[c].x, fmaf(v.y, b[c].y, fmaf(v.z, b[c].z, fmaf(v.w, b[c].w, acc[a][c]))));
        }
    }
}

// --------------------------------------------------------------- T and X
// One CTA per chunk and value head: tx[chunk] = T then X, 64 x 64 each.
template <typename E>
__global__ void __launch_bounds__(NT) delta_prep(const E* __restrict__ q, const E* __restrict__ k,
                                                 const float* __restrict__ g, const float* __restrict__ beta,
                                                 const int* __restrict__ lens, float* __restrict__ tx, Geo ge) {
    extern __shared__ __align__(16) float sm[];
    __shared__ Decays d;
    const int tid = threadIdx.x, c = blockIdx.x % ge.nc, bh = blockIdx.x / ge.nc;
    const int b = bh / ge.H, h = bh % ge.H, KH = ge.H / ge.G;
    const int n = min(row_len(lens, b, ge.T) - c * C, C);
    if (n <= 0) return;
    const int LK = ge.N + 4;
    float* sk = sm;
    float* sq = sk + C * LK;
    float* a = sq + C * LK;
    float* p = a + C * LT;
    float* w = p + C * LT;
    const int64_t t0 = (int64_t)b * ge.T + (int64_t)c * C;
    const int64_t ko = (t0 * KH + h / ge.G) * ge.N, ks = (int64_t)KH * ge.N;
    load_rows(sk, LK, k + ko, ks, C, ge.N, n, tid);
    load_rows(sq, LK, q + ko, ks, C, ge.N, n, tid);
    if (tid < 32) chunk_decays(d, g + t0 * ge.H + h, beta + t0 * ge.H + h, ge.H, n, tid);
    __syncthreads();
    const int ti = tid / 16, tj = tid % 16;
    float kk[4][4] = {}, qk[4][4] = {};
    mm_rr<4, 16, 16>(kk, sk, LK, sk, LK, ge.N, ti, tj);
    mm_rr<4, 16, 16>(qk, sq, LK, sk, LK, ge.N, ti, tj);
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int i = ti + 16 * x, j = tj + 16 * y;
            const float m = i >= j ? decay_between(d, i, j) : 0.f;
            a[i * LT + j] = i > j ? d.beta[i] * (m * kk[x][y]) : 0.f;
            p[i * LT + j] = i >= j ? m * qk[x][y] : 0.f;
        }
    __syncthreads();
    tri_inverse_in_place<LT>(a, w, tid);
    const float* t = a;
    float x[4][4] = {};
    mm_rk<4, 16>(x, p, LT, t, LT, C, ti, 4 * tj);
    float* out = tx + (int64_t)blockIdx.x * 2 * C * C;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = ti + 16 * r;
        *reinterpret_cast<float4*>(out + i * C + 4 * tj) = ld4(t + i * LT + 4 * tj);
        *reinterpret_cast<float4*>(out + C * C + i * C + 4 * tj) = make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
    }
}

// --------------------------------------------------------------- forward scan
// One CTA per value head and slice of PW state columns (they never mix),
// walking the chunks.  With `states`, the state entering each chunk and the
// writes U are kept for the gradients and no output is made.
template <typename E>
__global__ void __launch_bounds__(NT) delta_scan(const E* __restrict__ q, const E* __restrict__ k,
                                                 const E* __restrict__ v, const float* __restrict__ g,
                                                 const float* __restrict__ beta, const float* __restrict__ tx,
                                                 const float* h0, const int* __restrict__ lens, float scale,
                                                 E* __restrict__ o, float* h_final, float* __restrict__ states,
                                                 float* __restrict__ writes, Geo ge) {
    extern __shared__ __align__(16) float sm[];
    __shared__ Decays d;
    const int np = (ge.P + PW - 1) / PW;
    const int tid = threadIdx.x, p0 = (int)(blockIdx.x % np) * PW, bh = (int)(blockIdx.x / np);
    const int b = bh / ge.H, h = bh % ge.H, KH = ge.H / ge.G, N = ge.N, P = ge.P;
    const int len = row_len(lens, b, ge.T), LK = N + 4;
    float* kq = sm;                  // K rows then Q rows
    float* stx = kq + 2 * C * LK;    // T rows then X rows
    float* s = stx + 2 * C * LT;
    float* r = s + N * LS;
    float* u = r + C * LS;
    const int rg = tid / 8, c0 = 4 * (tid % 8);
    const int64_t so = (int64_t)bh * N * P;
    if (h0) {
        load_slice(s, h0 + so, P, N, p0, P, N, tid);
    } else {
        for (int e = tid; e < N * LS; e += NT) s[e] = 0.f;
    }
    for (int c = 0; c * C < len; ++c) {
        const int n = min(len - c * C, C);
        const int64_t t0 = (int64_t)b * ge.T + (int64_t)c * C;
        const int64_t ko = (t0 * KH + h / ge.G) * N, ks = (int64_t)KH * N;
        const int64_t ci = (int64_t)bh * ge.nc + c;
        __syncthreads();
        load_rows(kq, LK, k + ko, ks, C, N, n, tid);
        if (o) load_rows(kq + C * LK, LK, q + ko, ks, C, N, n, tid);
        load_rows(stx, LT, tx + ci * 2 * C * C, C, 2 * C, C, 2 * C, tid);
        load_slice(r, v + (t0 * ge.H + h) * P, (int64_t)ge.H * P, C, p0, P, n, tid);
        if (tid < 32) chunk_decays(d, g + t0 * ge.H + h, beta + t0 * ge.H + h, ge.H, n, tid);
        __syncthreads();
        if (states)
            for (int e = tid; e < N * PW; e += NT)
                if (p0 + e % PW < P) states[ci * N * P + (int64_t)(e / PW) * P + p0 + e % PW] = s[(e / PW) * LS + e % PW];
        float ks_[4][4] = {};
        mm_rk<4, 32>(ks_, kq, LK, s, LS, N, rg, c0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = rg + 32 * x;
#pragma unroll
            for (int y = 0; y < 4; ++y) r[i * LS + c0 + y] = d.beta[i] * (r[i * LS + c0 + y] - d.in[i] * ks_[x][y]);
        }
        __syncthreads();
        float ur[4][4] = {};
        mm_rk<4, 32>(ur, stx, LT, r, LS, C, rg, c0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = rg + 32 * x;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                u[i * LS + c0 + y] = d.out[i] * ur[x][y];
                if (p0 + c0 + y >= P) continue;
                if (writes) writes[ci * C * P + (int64_t)i * P + p0 + c0 + y] = ur[x][y];
                if (o && i < n)
                    o[((t0 + i) * ge.H + h) * P + p0 + c0 + y] =
                        from_f<E>(scale * (d.in[i] * ks_[x + 2][y] + ur[x + 2][y]));
            }
        }
        __syncthreads();
        if (4 * rg < N) {
            float ns[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) ns[x][y] = d.all * s[(4 * rg + x) * LS + c0 + y];
            mm_kr<4>(ns, kq, LK, u, LS, C, 4 * rg, c0);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) s[(4 * rg + x) * LS + c0 + y] = ns[x][y];
        }
    }
    __syncthreads();
    if (h_final)
        for (int e = tid; e < N * PW; e += NT)
            if (p0 + e % PW < P) h_final[so + (int64_t)(e / PW) * P + p0 + e % PW] = s[(e / PW) * LS + e % PW];
    if (o)
        for (int64_t e = tid; e < (int64_t)(ge.T - len) * PW; e += NT)
            if (p0 + (int)(e % PW) < P)
                o[(((int64_t)b * ge.T + len + e / PW) * ge.H + h) * P + p0 + e % PW] = from_f<E>(0.f);
}

// --------------------------------------------------------------- backward scan
// The same walk from the last chunk: the gradient of the state leaving each
// chunk is kept in `after`, Z in `zs`.
template <typename E>
__global__ void __launch_bounds__(NT) delta_back_scan(const E* __restrict__ q, const E* __restrict__ k,
                                                      const E* __restrict__ dout, const float* __restrict__ g,
                                                      const float* __restrict__ beta, const float* __restrict__ tx,
                                                      const float* dh, const int* __restrict__ lens, float scale,
                                                      float* gh0, float* __restrict__ after,
                                                      float* __restrict__ zs, Geo ge) {
    extern __shared__ __align__(16) float sm[];
    __shared__ Decays d;
    const int np = (ge.P + PW - 1) / PW;
    const int tid = threadIdx.x, p0 = (int)(blockIdx.x % np) * PW, bh = (int)(blockIdx.x / np);
    const int b = bh / ge.H, h = bh % ge.H, KH = ge.H / ge.G, N = ge.N, P = ge.P;
    const int len = row_len(lens, b, ge.T), LK = N + 4;
    float* kq = sm;
    float* stx = kq + 2 * C * LK;
    float* s = stx + 2 * C * LT;  // dS
    float* r = s + N * LS;        // scale dO, then scale e^G dO
    float* u = r + C * LS;        // e^{G_end - G} K dS, then -e^G beta Z
    const int rg = tid / 8, c0 = 4 * (tid % 8);
    const int64_t so = (int64_t)bh * N * P;
    if (dh) {
        load_slice(s, dh + so, P, N, p0, P, N, tid);
    } else {
        for (int e = tid; e < N * LS; e += NT) s[e] = 0.f;
    }
    for (int c = (len + C - 1) / C - 1; c >= 0; --c) {
        const int n = min(len - c * C, C);
        const int64_t t0 = (int64_t)b * ge.T + (int64_t)c * C;
        const int64_t ko = (t0 * KH + h / ge.G) * N, ks = (int64_t)KH * N;
        const int64_t ci = (int64_t)bh * ge.nc + c;
        __syncthreads();
        load_rows(kq, LK, k + ko, ks, C, N, n, tid);
        load_rows(kq + C * LK, LK, q + ko, ks, C, N, n, tid);
        load_rows(stx, LT, tx + ci * 2 * C * C, C, 2 * C, C, 2 * C, tid);
        load_slice(r, dout + (t0 * ge.H + h) * P, (int64_t)ge.H * P, C, p0, P, n, tid);
        if (tid < 32) chunk_decays(d, g + t0 * ge.H + h, beta + t0 * ge.H + h, ge.H, n, tid);
        __syncthreads();
        for (int e = tid; e < N * PW; e += NT)
            if (p0 + e % PW < P) after[ci * N * P + (int64_t)(e / PW) * P + p0 + e % PW] = s[(e / PW) * LS + e % PW];
        float w[2][4] = {};
        mm_rk<2, 32>(w, kq, LK, s, LS, N, rg, c0);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int i = rg + 32 * x;
                u[i * LS + c0 + y] = d.out[i] * w[x][y];
                r[i * LS + c0 + y] *= scale;
            }
        __syncthreads();
        float z[2][4] = {};
        mm_kr<2>(z, stx, LT, u, LS, C, 2 * rg, c0);
        mm_kr<2>(z, stx + C * LT, LT, r, LS, C, 2 * rg, c0);
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = 2 * rg + x;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float gvv = d.beta[i] * z[x][y];
                u[i * LS + c0 + y] = -d.in[i] * gvv;
                r[i * LS + c0 + y] *= d.in[i];
                if (p0 + c0 + y >= P) continue;
                zs[ci * C * P + (int64_t)i * P + p0 + c0 + y] = z[x][y];
            }
        }
        __syncthreads();
        if (4 * rg < N) {
            float ns[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) ns[x][y] = d.all * s[(4 * rg + x) * LS + c0 + y];
            mm_kr<4>(ns, kq, LK, u, LS, C, 4 * rg, c0);
            mm_kr<4>(ns, kq + C * LK, LK, r, LS, C, 4 * rg, c0);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) s[(4 * rg + x) * LS + c0 + y] = ns[x][y];
        }
    }
    __syncthreads();
    if (gh0)
        for (int e = tid; e < N * PW; e += NT)
            if (p0 + e % PW < P) gh0[so + (int64_t)(e / PW) * P + p0 + e % PW] = s[(e / PW) * LS + e % PW];
}

// --------------------------------------------------------------- dQ, dK, dV, dg, dbeta
// One CTA per chunk and value head.  gq and gk are the key heads' gradients
// when every value head has its own key head, else this value head's part in
// fp32, summed over the group by delta_sum_heads in a fixed order.
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
    float* pm = sq + C * LK;
    float* wm = pm + C * LT;
    float* sb = wm + C * LT;  // 32 rows of S, then of dS+
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
        mm_rr<4, 16, 16>(du, so, LP, su, LP, P, ti, tj);
        mm_rr<4, 16, 16>(zu, sz, LP, su, LP, P, ti, tj);
        mm_rr<4, 16, 16>(kk, sk, LK, sk, LK, N, ti, tj);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int i = ti + 16 * x;
            float gb = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int j = tj + 16 * y;
                const float m = i >= j ? decay_between(d, i, j) : 0.f;
                pm[i * LT + j] = i >= j ? scale * (m * du[x][y]) : 0.f;
                if (i > j) {
                    const float z = m * zu[x][y];
                    gb = fmaf(z, kk[x][y], gb);
                    wm[i * LT + j] = wm[j * LT + i] = -d.beta[i] * z;
                } else if (i == j) {
                    wm[i * LT + i] = 0.f;
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
        mm_rr<2, 32, 8>(aq, so, LP, sb, LP, P, rg, cg);
        mm_rr<2, 32, 8>(az, sz, LP, sb, LP, P, rg, cg);
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
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int i = rg + 32 * x;
            float qv[4], kv[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                qv[y] = scale * d.in[i] * aq[x][y];
                kv[y] = d.out[i] * au[x][y] - d.beta[i] * d.in[i] * az[x][y];
            }
            // (columns past N read the padding or the next row of sk; they are not kept)
            for (int j = 0; j < C; ++j) {
                const float p1 = pm[i * LT + j], p2 = pm[j * LT + i], p3 = wm[i * LT + j];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int col = min(nb + cg + 8 * y, N - 1);
                    qv[y] = fmaf(p1, sk[j * LK + col], qv[y]);
                    kv[y] = fmaf(p2, sq[j * LK + col], fmaf(p3, sk[j * LK + col], kv[y]));
                }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int col = nb + cg + 8 * y;
                if (col >= N) continue;
                qgq[x] = fmaf(sq[i * LK + col], qv[y], qgq[x]);
                kz[x] = fmaf(sk[i * LK + col], az[x][y], kz[x]);
                kus = fmaf(d.out[i] * sk[i * LK + col], au[x][y], kus);
                if (i < n) {
                    gq[go + i * gs + col] = from_f<O>(qv[y]);
                    gk[go + i * gs + col] = from_f<O>(kv[y]);
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
size_t tx_floats(const DeltaArgs& a) { return (size_t)(a.Bz * a.H * chunks(a)) * 2 * C * C; }
size_t state_floats(const DeltaArgs& a) { return (size_t)(a.Bz * a.H * chunks(a)) * a.N * a.P; }
size_t write_floats(const DeltaArgs& a) { return (size_t)(a.Bz * a.H * chunks(a)) * C * a.P; }
size_t part_floats(const DeltaArgs& a) { return a.H == a.KH ? 0 : (size_t)(a.Bz * a.T * a.H) * a.N; }

template <typename F>
cudaError_t allow_smem(F* f, size_t bytes) {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(f), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

Geo geo(const DeltaArgs& a) {
    return Geo{(int)a.T, (int)a.H, (int)(a.H / a.KH), (int)a.N, (int)a.P, (int)chunks(a)};
}
size_t scan_smem(const DeltaArgs& a) { return sizeof(float) * (2 * C * (a.N + 4) + 2 * C * LT + a.N * LS + 2 * C * LS); }

template <typename E>
cudaError_t prep(const DeltaArgs& a, float* tx, cudaStream_t st) {
    const size_t sm = sizeof(float) * (2 * C * (a.N + 4) + 2 * C * LT + 32 * 32);
    cudaError_t e = allow_smem(delta_prep<E>, sm);
    if (e != cudaSuccess) return e;
    delta_prep<E><<<(unsigned)(a.Bz * a.H * chunks(a)), NT, sm, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), a.g, a.beta, a.lens, tx, geo(a));
    return cudaGetLastError();
}

template <typename E>
cudaError_t scan(const DeltaArgs& a, const float* tx, void* o, float* h_final, float* states, float* writes,
                 cudaStream_t st) {
    const size_t sm = scan_smem(a);
    cudaError_t e = allow_smem(delta_scan<E>, sm);
    if (e != cudaSuccess) return e;
    delta_scan<E><<<(unsigned)((a.P + PW - 1) / PW * a.Bz * a.H), NT, sm, st>>>(
        static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.v), a.g, a.beta, tx, a.h0, a.lens,
        a.scale, static_cast<E*>(o), h_final, states, writes, geo(a));
    return cudaGetLastError();
}

template <typename E>
cudaError_t forward(const DeltaArgs& a, void* ws, cudaStream_t st) {
    float* tx = static_cast<float*>(ws);
    cudaError_t e = prep<E>(a, tx, st);
    return e != cudaSuccess ? e : scan<E>(a, tx, a.o, a.h_final, nullptr, nullptr, st);
}

template <typename E, typename O>
cudaError_t grad(const DeltaArgs& a, const float* states, const float* after, const float* writes, const float* zs,
                 void* gq, void* gk, cudaStream_t st) {
    const size_t sm = sizeof(float) * (3 * C * (a.P + 4) + 2 * C * (a.N + 4) + 2 * C * LT + 32 * (a.P + 4));
    cudaError_t e = allow_smem(delta_grad<E, O>, sm);
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
    float* rest = pk + part_floats(a);  // T and X; the tensor-core kernels' own
    cudaError_t e;
    if constexpr (TC) {
        e = launch_back_scans_tc(a, rest, states, after, writes, zs, st);
    } else {
        e = prep<E>(a, rest, st);
        if (e == cudaSuccess) e = scan<E>(a, rest, nullptr, nullptr, states, writes, st);
        const size_t sm = scan_smem(a);
        if (e == cudaSuccess) e = allow_smem(delta_back_scan<E>, sm);
        if (e != cudaSuccess) return e;
        delta_back_scan<E><<<(unsigned)((a.P + PW - 1) / PW * a.Bz * a.H), NT, sm, st>>>(
            static_cast<const E*>(a.q), static_cast<const E*>(a.k), static_cast<const E*>(a.dout), a.g, a.beta, rest,
            a.dh_final, a.lens, a.scale, a.gh0, after, zs, geo(a));
        e = cudaGetLastError();
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
    return a.dtype == CSSD_F32 ? sizeof(float) * delta::tx_floats(a) : delta::tc_workspace_bytes(a);
}
size_t delta_backward_workspace_bytes(const DeltaArgs& a) {
    return sizeof(float) * (2 * delta::state_floats(a) + 2 * delta::write_floats(a) + 2 * delta::part_floats(a)) +
           (a.dtype == CSSD_F32 ? sizeof(float) * delta::tx_floats(a) : delta::tc_back_bytes(a));
}

cudaError_t launch_delta_forward(const DeltaArgs& a, void* ws, cudaStream_t st) {
    return a.dtype == CSSD_F32 ? delta::forward<float>(a, ws, st) : delta::launch_forward_tc(a, ws, st);
}
cudaError_t launch_delta_backward(const DeltaArgs& a, void* ws, cudaStream_t st) {
    if (a.dtype == CSSD_BF16) return delta::backward<__nv_bfloat16>(a, ws, st);
    if (a.dtype == CSSD_F16) return delta::backward<__half>(a, ws, st);
    return delta::backward<float>(a, ws, st);
}

}  // namespace cssd
