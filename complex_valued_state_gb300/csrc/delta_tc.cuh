// What the tensor-core kernels of the gated delta rule share: operands in
// IEEE half with a power-of-two scale a row, the chunk image that the prep
// kernel leaves for the scans, and waits that give up.
//
// Precision.  A 16-bit input row times its power of two is exact in half (11
// bits hold bf16's 8 and half's own 11; what lies 2^-37 below the row's
// largest value is dropped).  An intermediate is held as two halves, hi (the
// value rounded to 11 bits) and lo (the remainder, at most 2^-12 of it, rounded
// to 11 bits): 2^-24 of the row's largest value.  A product of an exact operand
// with a split one takes two passes, of two split ones three (lo lo is left
// out, 2^-24), all into one fp32 accumulator, the low parts first: the
// accumulator drops what lies below its last bit at every step, and so only the
// last pass does at the full value.  The states, which are float32 tensors of
// the interface, keep fp32 accuracy.
#pragma once

#include "delta_common.cuh"
#include "pairs.cuh"
#include "tcgen05.cuh"

namespace cssd {
namespace delta {

constexpr long long kDeltaWait = 4000000000LL;  // ~2 s at 2 GHz

// The power of two that brings `top` (a row's largest absolute value) into
// [2^13, 2^14), and its inverse.  An infinite or NaN top gives a scale whose
// products are infinite or NaN again.
struct RowScale {
    float up, down;
};
__device__ __forceinline__ RowScale row_scale(float top) {
    int e = (int)((__float_as_uint(top) >> 23) & 255u);
    e = max(e, 14);
    return {__uint_as_float((uint32_t)(267 - e) << 23), __uint_as_float((uint32_t)(e - 13) << 23)};
}

__device__ __forceinline__ uint32_t pack2(float x0, float x1) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x1), "f"(x0));
    return r;
}
__device__ __forceinline__ float2 halves(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// Two values (already scaled) as half pairs: element 0 in the low half.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    hi = pack2(x0, x1);
    const float2 h = halves(hi);
    lo = pack2(x0 - h.x, x1 - h.y);
}

// A pair of 16-bit inputs as floats.
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Largest absolute value of packed pairs, as packed 16-bit patterns (for both
// types the order of |x| is that of the bits; NaN is above infinity).
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
    return __vmaxu2(a & 0x7FFF7FFFu, b & 0x7FFF7FFFu);
}
template <typename E>
__device__ __forceinline__ float top_of(uint32_t m) {
    const float2 f = unpack2(m, E());
    return f.x != f.x || f.y != f.y ? __uint_as_float(0x7F800000u) : fmaxf(f.x, f.y);
}

// D[tmem] (+)= A[tmem] B[smem]^T, half operands.  Row m of A is lane m; K
// elements 2c and 2c + 1 are the halves of column c.  Called by a converged
// warp, one elected lane issuing, so that the operands stay warp-uniform (58
// cycles an MMA when a single diverged lane issued them, against 34 the pipe
// needs at N = 64).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t.reg .b64 b;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
        : "memory");
}
// The elected lane's commit (the same lane: election picks one lane of a mask).
__device__ __forceinline__ void commit_elected(uint64_t* m) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(tc::smem_u32(m))
        : "memory");
}

__device__ __forceinline__ f2 raw2(uint32_t a, uint32_t b) { return mk2(__uint_as_float(a), __uint_as_float(b)); }

// Register shares of the warpgroups (multiples of 8; together at most what
// the block was launched with).
template <int R>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// 32 TMEM lanes (this warp's quarter) x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// 16 bytes into shared memory, or zeros where there is nothing to read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
// An arrival (counted in the barrier's expected ones) once this thread's
// copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* m) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(m)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Bulk copy of `bytes` (a multiple of 16; both addresses 16-byte aligned) from
// this CTA's shared memory, in the thread's current bulk group.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
// `bytes` (a multiple of 16) from a 16-byte aligned address into L2.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until shared memory of the thread's bulk groups may be written again / until they are complete.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int R, int FROM>
__device__ __forceinline__ void set_registers() {
    if constexpr (R > FROM) more_registers<R>();
    if constexpr (R < FROM) fewer_registers<R>();
}
// A pair rounded to 16-bit values, element 0 in the low half.
template <typename E>
__device__ __forceinline__ uint32_t pack_as(f2 v) {
    float a, b;
    uint32_t r;
    un2(v, a, b);
    if constexpr (sizeof(E) == 2 && !__is_same(E, __half))
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Registers into 32 TMEM lanes x 8 consecutive columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* m) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(m)) : "memory");
}

// Wait for a phase parity; false once this or another wait of the CTA has
// given up (after ~2 s), which `gave_up` tells the others.
__device__ __forceinline__ bool wait_or_give_up(uint64_t* m, uint32_t parity, volatile int* gave_up) {
    if (tc::mbar_try_wait(m, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (tc::mbar_try_wait(m, parity)) return true;
        if (*gave_up) return false;
        if (clock64() - t0 > kDeltaWait) {
            *gave_up = 1;
            return false;
        }
    }
}

// The same by a whole warp: true for all its lanes or for none.
__device__ __forceinline__ bool warp_wait(uint64_t* m, uint32_t parity, volatile int* gave_up) {
    return __all_sync(0xffffffffu, wait_or_give_up(m, parity, gave_up));
}

// e^{G_i - G_j} for i >= j as e[i] f[i / 16][j], a product over the start of
// i's block of 16 tokens (so that a table of 256 exponentials serves a chunk):
// exact to fp32 rounding while a block's decay, which f undoes, stays above
// e^-40; `steep` is set where it does not.  `down` (may be null) multiplies f.
// 256 threads.
struct DecayTables {
    float f[4][C], e[C];
    int steep;  // zeroed by the caller, a barrier before
};
__device__ __forceinline__ void decay_tables(DecayTables& t, const Decays& d, const float* down, int tid) {
    const int a = 16 * (tid / C), j = tid % C;
    // G_a - G_j as a float and what its rounding leaves
    const float at = d.hi[a] - d.hi[j], back = at - d.hi[a];
    const float rest = ((d.hi[a] - (at - back)) - (d.hi[j] + back)) + (d.lo[a] - d.lo[j]);
    t.f[tid / C][j] = j < a + 16 ? expf(at) * (1.f + rest) * (down ? down[j] : 1.f) : 0.f;
    if (j / 16 == tid / C) {
        t.e[j] = expf(-at) * (1.f - rest);
        if (!(fabsf(at) < 40.f)) t.steep = 1;  // (a NaN or infinite sum too)
    }
}
// The same directly (exp's own error is relative to a value that falls as
// fast as its argument grows).
__device__ __forceinline__ float steep_decay(const Decays& d, int i, int j) {
    return __expf((d.hi[i] - d.hi[j]) + (d.lo[i] - d.lo[j]));
}

// What a chunk's prep leaves in the workspace, copied whole into shared memory
// by the scans.  Per value head an image: [T; X] (the backward scan: [T^T;
// X^T]) as a B operand of 128 rows (T's 64, then X's) by 64, hi then lo, and
// the per-token factors the scan multiplies by.  Per key head the operands of
// K and Q, below.
struct Image {
    static constexpr uint32_t SBO = 128, LBO = 16 * 128;  // row groups, column groups of 8
    static constexpr uint32_t PART = 8 * LBO;              // one part's bytes
    static constexpr uint32_t F = 2 * PART;                // floats from here
    // Forward (T and X times beta): of the state's answer in R, of the products
    // in U and in U', of the two parts of o.
    static constexpr int KB = 0, UU = 64, UW = 128, OQ = 192, OX = 256;
    // Backward: of K dS in the first operand W, of the two products in Z, of Z
    // in the second operand, of dO in the third.
    static constexpr int WK = 0, ZT = 64, ZX = 128, RZ = 192, DQ = 256;
    // exp(G_end); and what bounds the scan's operands (see delta_scan_tc).
    static constexpr int ALL = 320, BND1 = 321, BND2 = 322, BND3 = 323;
    // Backward: the inverse scales of K's and Q's rows.
    static constexpr int KD = 324, QD = 388, FLOATS = 452;
    static constexpr uint32_t BYTES = F + 4 * FLOATS;
    static constexpr uint32_t STRIDE = (BYTES + 255) / 256 * 256;
};
// [Q; K]: rows i (64 of Q, then 64 of K) by ND; a row group's columns are
// contiguous, so each of the two is.
template <int ND>
struct QK {
    static constexpr uint32_t LBO = 128, SBO = (ND / 8) * LBO, KROWS = 8 * SBO, BYTES = 2 * KROWS;
};
// K^T, then (the backward) Q^T: rows k (ND) by 64 tokens.
template <int ND>
struct KT {
    static constexpr uint32_t SBO = 128, LBO = (ND / 8) * SBO, BYTES = 8 * LBO;
};
template <int ND>
struct Operands {
    static constexpr uint32_t KT0 = QK<ND>::BYTES, QT0 = KT0 + KT<ND>::BYTES;
    static constexpr uint32_t FWD = QT0, BWD = QT0 + KT<ND>::BYTES;  // bytes the two directions leave
};

}  // namespace delta
}  // namespace cssd
