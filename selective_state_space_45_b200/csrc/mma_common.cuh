// mma_common.cuh -- warp-level matrix products on registers (mma.sync m16n8k16, bf16 in,
// fp32 out), the shared-memory fragment loads that feed them, and fp32 operands as sums of
// bf16 pieces.
//
// Fragment layouts, lane = 4 g + t (g = 0..7, t = 0..3): an accumulator tile [16 x 8] holds
// (row g, columns 2t, 2t+1) in c[0], c[1] and (row g + 8, the same columns) in c[2], c[3].
// Two neighbouring accumulator tiles are, once converted, one A operand [16 x 16]: that is
// what lets a chain of products stay in registers.
#pragma once

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
__device__ __forceinline__ void stsm4_t(unsigned addr, const unsigned (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// The pair (x, y) as `NP` packed bf16 pairs whose sums give them back.  Every piece but the
// last is cut off (the upper 16 bits as they are), so the remainder is exact; three pieces
// hold all 24 bits of an fp32 value.  A last piece of one or two is rounded to nearest:
// 2^-9 and 2^-17 of the value at most.
template <int NP> __device__ __forceinline__ void split_pair(float x, float y, unsigned (&p)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        if (i == NP - 1 && NP < 3) {
            p[i] = pack_bf16x2(x, y);
        } else {
            p[i] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
            if (i < NP - 1) {
                const float2 r = fadd2(f2(x, y), f2(-__uint_as_float(__float_as_uint(x) & 0xffff0000u),
                                                    -__uint_as_float(__float_as_uint(y) & 0xffff0000u)));
                x = r.x; y = r.y;
            }
        }
    }
}

// Two neighbouring accumulator tiles as the pieces of one A operand.
template <int NP>
__device__ __forceinline__ void split_tiles(const float (&lo)[4], const float (&hi)[4], unsigned (&a)[NP][4]) {
    unsigned p[NP];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float *c = (r & 2) ? hi : lo;
        split_pair<NP>(c[2 * (r & 1)], c[2 * (r & 1) + 1], p);
#pragma unroll
        for (int i = 0; i < NP; ++i) a[i][r] = p[i];
    }
}

__device__ __forceinline__ void zero4(float (&c)[4]) { c[0] = c[1] = c[2] = c[3] = 0.f; }

// 16-byte asynchronous copy, or 16 zero bytes when !ok (the source is then not read).
__device__ __forceinline__ void cp_async_16z(unsigned smem_dst, const void *gmem_src, bool ok) {
    const int n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_dst), "l"(gmem_src), "r"(n) : "memory");
}

}  // namespace ssm
