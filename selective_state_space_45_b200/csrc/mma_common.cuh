// mma_common.cuh -- warp-level matrix products on registers (mma.sync m16n8k16, bf16 or fp16
// in, fp32 out), the shared-memory fragment loads that feed them, and fp32 operands as sums
// of bf16 or fp16 pieces.
//
// Fragment layouts, lane = 4 g + t (g = 0..7, t = 0..3): an accumulator tile [16 x 8] holds
// (row g, columns 2t, 2t+1) in c[0], c[1] and (row g + 8, the same columns) in c[2], c[3].
// Two neighbouring accumulator tiles are, once converted, one A operand [16 x 16]: that is
// what lets a chain of products stay in registers.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace ssm {

__device__ __forceinline__ void mma_bf16(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned smem_u32(const void *p) {
    return static_cast<unsigned>(__cvta_generic_to_shared(p));
}

// Four 8x8 bf16 tiles; lanes 8i..8i+7 give the row addresses of tile i (16-byte aligned).
// Lane 4g+t receives (row g, columns 2t, 2t+1) of each tile, or with _t of its transpose.
__device__ __forceinline__ void ldsm4(unsigned (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(unsigned (&r)[4], unsigned addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4(unsigned addr, const unsigned (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void stsm4_t(unsigned addr, const unsigned (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// The pair (x, y) as three packed bf16 pairs whose sums give all 24 bits of each back: every
// piece is cut off (the upper 16 bits as they are), so the remainders are exact.
__device__ __forceinline__ void split_bf16(float x, float y, unsigned (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
        if (i < 2) {
            const float2 r = ffma2(f2(__uint_as_float(__float_as_uint(x) & 0xffff0000u),
                                      __uint_as_float(__float_as_uint(y) & 0xffff0000u)), f2(-1.f, -1.f), f2(x, y));
            x = r.x; y = r.y;
        }
    }
}

// fp16 operands.  An fp32 value times a power of two c goes in as one fp16 value, or as two
// whose sum keeps 22 bits or more of it; c puts the largest magnitude of the tile between
// 2^13 and 2^14, so that nothing overflows and what falls below fp16's smallest step is under
// 2^-38 of the largest.
__device__ __forceinline__ void mma_f16(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&h);
}

// The power of two c for values whose largest magnitude has the bits `m` (as an integer), and
// its inverse.  Of an infinite one the inverse is NaN: beside it the other values vanish, and a
// product without them must not look like a result.
struct Pow2 { float c, inv; };
constexpr unsigned kNanBits = 0x7fffffffu;
__device__ __forceinline__ Pow2 pow2_for(unsigned m) {
    const unsigned f = min(267u - (m >> 23), 253u);
    return {__uint_as_float(f << 23), __uint_as_float(m >= 0x7f800000u ? kNanBits : (254u - f) << 23)};
}
__device__ __forceinline__ unsigned warp_max_bits(float m) {
    return __reduce_max_sync(0xffffffffu, __float_as_uint(m));      // m >= 0: ordered as integers
}

template <int NP> __device__ __forceinline__ void split_f16(float2 x, float c, unsigned (&p)[NP]) {
    static_assert(NP == 1 || NP == 2);
    x = fmul2(x, f2(c, c));
    p[0] = pack_f16x2(x.x, x.y);
    if constexpr (NP == 2) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&p[0]));
        const float2 r = ffma2(h, f2(-1.f, -1.f), x);
        p[1] = pack_f16x2(r.x, r.y);
    }
}

// Two neighbouring accumulator tiles, rows g times c0 and rows g + 8 times c1, as the pieces of
// one A operand.
template <int NP>
__device__ __forceinline__ void split_tiles(const float (&lo)[4], const float (&hi)[4], float c0, float c1, unsigned (&a)[NP][4]) {
    unsigned p[NP];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float *x = (r & 2) ? hi : lo;
        split_f16<NP>(f2(x[2 * (r & 1)], x[2 * (r & 1) + 1]), r & 1 ? c1 : c0, p);
#pragma unroll
        for (int i = 0; i < NP; ++i) a[i][r] = p[i];
    }
}

template <int NP>
__device__ __forceinline__ void split_tiles(const float (&lo)[4], const float (&hi)[4], float c, unsigned (&a)[NP][4]) {
    split_tiles<NP>(lo, hi, c, c, a);
}

// acc += A B over pieces, the product of two second pieces left out (2^-22 of the leading
// one and below), the small products first.
template <int PA, int PB>
__device__ __forceinline__ void mma_pieces(float (&acc)[4], const unsigned (&a)[PA][4], const unsigned (&b)[PB][4], int tile) {
    if constexpr (PA == 2) mma_f16(acc, a[1], b[0][2 * tile], b[0][2 * tile + 1]);
    if constexpr (PB == 2) mma_f16(acc, a[0], b[1][2 * tile], b[1][2 * tile + 1]);
    mma_f16(acc, a[0], b[0][2 * tile], b[0][2 * tile + 1]);
}

__device__ __forceinline__ void zero4(float (&c)[4]) { c[0] = c[1] = c[2] = c[3] = 0.f; }

// 16-byte asynchronous copy, or 16 zero bytes when !ok (the source is then not read).
__device__ __forceinline__ void cp_async_16z(unsigned smem_dst, const void *gmem_src, bool ok) {
    const int n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_dst), "l"(gmem_src), "r"(n) : "memory");
}

}  // namespace ssm
