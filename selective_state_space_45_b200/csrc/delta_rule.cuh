// delta_rule.cuh -- the gated delta rule by chunks of 32 tokens, the state in registers.
//
// Per sequence and head, with the headdim x dstate fp32 state S (dv = headdim rows, dk =
// dstate columns):
//     S' = exp(a_t) S,  e_t = v_t - S' k_t,  S = S' + beta_t e_t k_t^T,  y_t = scale S q_t
// Over a chunk of C tokens with start state S, r(t,s) = exp(a_{s+1} + ... + a_t),
// gam_t = r(t, before the chunk), end_s = r(last, s):
//     R_t = v_t - gam_t S k_t
//     e   = R - G (beta R),   G = (I + A diag(beta))^-1 A,   A(t,s) = r(t,s) (k_t.k_s) for s < t
//     y_t = scale gam_t S q_t + sum_{s<=t} Pm(t,s) beta_s e_s,  Pm(t,s) = scale r(t,s) (q_t.k_s)
//     S  <- gam_last S + sum_s (end_s beta_s e_s) k_s^T
// Every row of S (one value of headdim) goes through this on its own, given k, q, G and Pm,
// so a warp owns 16 rows and keeps them in registers as accumulator tiles [16 x dstate]:
// the state enters each product as a register operand and no step of the chain goes through
// shared memory or waits for another warp.  What depends on k, q, a and beta alone (G, Pm and
// the decays) is formed for all chunks in parallel by delta_prep_kernel, one warp per chunk,
// which also lays the chunk's k and q out as the chains' operands.  The warps of a CTA take
// turns at starting the copies of a later chunk (cp.async.bulk, cp.async for the rows of v,
// which one bulk copy each would take 70 cycles to start; two or three stages, mbarriers both
// ways) and otherwise wait for data only, never for each other.  Copying and converting the
// rows in the chains instead cost 1100 of 3700 cycles a chunk; a fifth warp for the copies
// costs the others the registers that they need (168 instead of 255: spills).
//
// What bounds it.  bf16, dstate 128: a chunk takes 2.0 us in a CTA that has its SM to itself and
// 3.6 us where two share one; 8 x 2048 tokens x 24 heads of 64 x 128 (192 CTAs) 226 us, and the
// prep kernel 102 us (75% of HBM's copy rate: it writes the blocks and the operands).  Alone, the
// mma.sync pipe is active for 51% of the time and half of the warps' cycles go to the fixed
// latencies of dependent instructions.  Two warps on a scheduler overlap those, but then meet in
// the pipe (59% active, a fifth of the cycles waiting for it; the products of a chunk come in
// bursts), which is most of the 1.8.  Shared memory (48% of its wavefronts) and HBM are not it.
// mma.sync rather than tcgen05 was chosen to keep the state and its products in registers with
// the warp that needs them next; the other has not been measured.
//
// The reverse pass runs the same chain backwards on the state's gradient dS, with dO = dy:
//     rhs = end (dS k) + Pm^T dO,  du = rhs - G^T (beta rhs),  dv = w = beta du,
//     dS <- gam_last dS + (scale gam dO) q^T - (gam w) k^T
//
// Precision: the products run on the tensor cores in fp16 with fp32 accumulation, every
// operand scaled by a power of two: one per token for k, one per chunk for q and the triangles,
// one per row and chunk for the state and what follows from it, each from the operand's own
// largest value.  With l_t the power of two that key t is scaled by, the triangles are those of
// the keys k_t / l_t with steps beta_t l_t^2, which no ratio of lengths spreads; l_t goes onto
// the tokens' vectors on either side of them.  (Bounds from the factors' largest values in
// place of the operands' own left 2e-2 of the state at keys 300 times as long as their
// neighbours, one scale for a chunk's keys 1e-3 at lengths spread over 10^6.)  Rows of headdim
// never meet, in range no more than in value: a row's inf or NaN stays in its row.  bf16
// inputs are then exact; fp32 operands go in as two fp16 values (22 bits or more), whatever
// the type of y: one behind a bf16 y made 11% of its values round the other way (8 x 2048
// tokens x 24 heads of 64 x 128: 280 us with the call, 312 with two).  The product of two second
// pieces is left out.  An fp32 y and state then come out at 5e-7 of the definition in 64 bits,
// gradients at 8e-7, where torch's fp32 products give 2e-7 and 4e-7.  Three bf16 pieces hold
// the same bits but cost half as many products again; two bf16 pieces gave 6e-6.
#pragma once

#include <type_traits>

#include "mma_common.cuh"
#include "tc_common.cuh"

namespace ssm {

struct DeltaArgs {
    const void *q, *k;      // prep kernel: [batch][seqlen][qk_heads][dstate]
    unsigned char *prep;    // [batch][heads][chunks] blocks of the prep kernel
    unsigned char *rows;    // [batch][qk_heads][chunks] k and q as operands, from the prep kernel
    unsigned *timeouts;     // counts waits that gave up
    const void *v;          // [batch][seqlen][heads][headdim]; the reverse pass: dy
    const float *a, *beta;  // [batch][seqlen][heads]
    void *y;                // forward: y; reverse pass: dv
    const float *h0;        // start state (reverse pass: the final state's gradient) or NULL
    float *hN;              // end state (reverse pass: the start state's gradient) or NULL
    // The backward's scratch.  A "part" is a warp's 16 rows: part = slice * warps + warp.  The last
    // kernel takes scaled fp16 operands, tiles of its shared memory as they stand, in two pieces
    // (one of a bf16 dy): e, w and dy of a part and chunk, and of a part and 32 columns the state
    // and its gradient at every boundary of 64 tokens (the first has no gradient, the end no state).
    unsigned char *e16, *w16, *y16;     // [batch][heads][chunks][parts][pieces] 16 rows of 32 tokens
    unsigned char *s16, *d16;           // [batch][heads][boundaries][dstate / 32][parts][pieces] 16 rows of 32 columns
    unsigned *smax;         // [batch][heads][boundaries][parts] largest |S| (reverse pass: |dS|), as bits
    unsigned *emax, *ymax;  // [batch][heads][chunks][parts] largest |e| (reverse pass: |w|) and, in the
                            // reverse pass, |dy|
    // Segments of a long sequence with few heads: chunks per segment, and per segment
    // [batch][heads][segments] the end state from a zero start (the first: from h0), later the next
    // one's start state, and the map that takes a start state's rows to their part of the end state.
    // Reverse passes: the same from the other end, gradients of start states.
    int seg_chunks;
    float *seg_state, *seg_map;     // [headdim][dstate], [dstate][dstate]
    bool end_slot;                  // the end state goes to the last segment's slot of seg_state, not hN
    int batch, seqlen, heads, qk_heads, P, N, slices;
    float scale;
};

constexpr int kDeltaC = 32;          // tokens per chunk
constexpr int kDeltaSave = 64;       // tokens between the states kept for the backward
constexpr int kTri = 512;            // bytes of a 16 x 16 tile of 16-bit values, rows of 32
constexpr int kOutRow = 48;          // bytes per row of a warp's output tile

// Byte offset of the 16-byte half `c` of row r in such a tile: the halves change places every
// four rows, so that eight rows' halves are eight different bank groups (ldmatrix).
__device__ __forceinline__ int tri_at(int r, int c) { return r * 32 + ((c ^ (r >> 2)) & 1) * 16; }

// What the prep kernel leaves per chunk and head.  A triangle is the three 16 x 16 tiles
// (0,0), (1,0), (1,1) per fp16 piece, scaled by a power of two: G and Pm, two pieces each.
// Vectors over the chunk's tokens, the scales of k and q (ck, cq) taken back out where a
// product with them is used:
enum {
    kVecGk,        // gam / ck: S k -> gam S k
    kVecSgq,       // scale gam / cq
    kVecBeta,
    kVecEk,        // end / ck
    kVecEbk,       // end beta / ck
    kVecBl,        // beta l
    kVecL,         // l = 2^13 / ck
    kVecScalars,   // then the scalars below
    kVecs
};
enum { kGamLast, kInvQ, kInvG, kInvP };           // the chunk's decay, 1 / scales of q, G and Pm
struct DeltaBlock {
    static constexpr int OFF_P = 6 * kTri, OFF_VEC = OFF_P + 6 * kTri, BYTES = OFF_VEC + kVecs * kDeltaC * 4;
};

// k and q of a chunk as the chains read them: scaled fp16, KP pieces of k, then of q, each 32
// rows of NP values (zeros past dstate and seqlen) padded by 16 bytes against bank conflicts.
template <int NP, int KP> struct DeltaRows {
    static constexpr int ROW = NP * 2 + 16, PIECE = kDeltaC * ROW, BYTES = 2 * KP * PIECE;
};

// A 16-bit tile of a part: 16 rows of 64 bytes (32 tokens, or 32 columns of the state).  The
// 16-byte quarters of a row change places with the row, so that eight rows' quarters of one
// column are eight bank groups (ldmatrix).
constexpr int kTok16 = 1024;
__device__ __forceinline__ int tok16_at(int r, int n) { return r * 64 + ((n ^ (r >> 1)) & 3) * 16; }

constexpr long long kDeltaWaitCycles = 2000000000LL;        // a bounded wait's limit, about a second

// NP: dstate rounded up; NW: warps with 16 rows each.  KP: pieces of q and k.  MODE 0:
// forward (y); 1: the forward again for the backward (e and the kept states); 2: the reverse pass; 3:
// a segment's end state and map (the recurrence of the identity's rows with v = 0); 4: the
// reverse of 3, a segment's gradient of its start state (its map is the forward's, transposed).
template <int NP_, int NW_, int KP_, typename Tv_, typename Tout_, int MODE_> struct DeltaCfg {
    static constexpr int NP = NP_, NW = NW_, MODE = MODE_, KP = KP_;
    using Tv = Tv_;        // v, or dy in the reverse pass
    using Tout = Tout_;
    static constexpr int C = kDeltaC, NT = 32 * NW;
    static constexpr int CTAS = KP == 1 && sizeof(Tv) == 2 ? 2 : 1;       // per SM
    static constexpr int PV = sizeof(Tv) == 4 ? 2 : 1;                        // pieces of v (dy)
    using Block = DeltaBlock;
    using Rows = DeltaRows<NP, KP>;
    static constexpr int KROW = Rows::ROW;
    static constexpr int VROW = NW * 16 * int(sizeof(Tv)) + 16;
    static constexpr int PIECE = Rows::PIECE;
    static constexpr int OFF_K = 0, OFF_Q = KP * PIECE, OFF_TRI = Rows::BYTES;
    static constexpr int OFF_V = OFF_TRI + Block::BYTES, STAGE = OFF_V + C * VROW;
    static constexpr bool BWD = MODE == 1 || MODE == 2;
    static constexpr int STAGES = KP == 1 ? 3 : 2;                        // three where two CTAs still fit
    static constexpr int OFF_BAR = STAGES * STAGE;                                 // mbarriers: full, empty
    static constexpr int OFF_OUT = OFF_BAR + 64;                              // per-warp output tiles
    static constexpr int OUT = BWD ? 2 * kTok16 : 1024;                       // bytes of a warp's tile
    static constexpr int SMEM_BYTES = OFF_OUT + NW * OUT;
};

// acc += A B of operands in KP bf16 pieces (1: exact, 3: all bits of fp32), the products of
// pieces below 2^-24 of the leading one left out.
template <int KP>
__device__ __forceinline__ void mma_exact(float (&acc)[4], const unsigned (&a)[KP][4], const unsigned (&b)[KP][4], int tile) {
#pragma unroll
    for (int i = KP - 1; i >= 0; --i)
#pragma unroll
        for (int j = KP - 1 - i; j >= 0; --j) mma_bf16(acc, a[i], b[j][2 * tile], b[j][2 * tile + 1]);
}

// One warp per chunk and head forms the chunk's block; the first head of each key head also
// writes the chunk's k and q as operands.  Four warps per CTA, each with its own scratch.
template <int NP, typename Tin> struct PrepScratch {
    static constexpr int RATROW = 33, NROW = 36, ROW = NP * int(sizeof(Tin)) + 16;
    float ck[kDeltaC];                                          // the keys' scales
    union {
        unsigned char rows[2][kDeltaC * ROW];                   // k and q as they come
        struct {
            unsigned char block[DeltaBlock::BYTES];               // as it goes out
            float at[kDeltaC * NROW];                           // at[s][t] = A(t, s)
            float rat[kDeltaC * RATROW + 4];                    // rat[t][s + 1] = r(t, s); later parts of G
            float beta[kDeltaC];                                // beta l^2
        };
    };
};

template <int NP, typename Tin>
__global__ void __launch_bounds__(128) delta_prep_kernel(const DeltaArgs p) {
    using Block = DeltaBlock;
    using Scratch = PrepScratch<NP, Tin>;
    constexpr int C = kDeltaC, RATROW = Scratch::RATROW, NROW = Scratch::NROW, ROW = Scratch::ROW;
    constexpr int KP = sizeof(Tin) == 4 ? 3 : 1, OP = sizeof(Tin) == 4 ? 2 : 1;      // pieces here, and as operands
    using Rows = DeltaRows<NP, OP>;
    extern __shared__ __align__(128) unsigned char delta_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int nchunk = (p.seqlen + C - 1) / C;
    const long long id = (long long)blockIdx.x * 4 + warp;      // head fastest: neighbours share q and k rows
    if (id >= (long long)p.batch * p.heads * nchunk) return;
    const int h = int(id % p.heads);
    const long long bc = id / p.heads;
    const int c = int(bc % nchunk), b = int(bc / nchunk);
    const int group = p.heads / p.qk_heads, hk = h / group, t0 = c * C;
    Scratch &sc = reinterpret_cast<Scratch *>(delta_smem)[warp];

    // the chunk's rows, all on their way at once
    {
        constexpr int E = 16 / sizeof(Tin), CR = NP / E;
        const size_t krow = size_t(p.qk_heads) * p.N;
        const size_t k0 = (size_t(b) * p.seqlen + t0) * krow + size_t(hk) * p.N;
        const Tin *kp = static_cast<const Tin *>(p.k) + k0, *qp = static_cast<const Tin *>(p.q) + k0;
        const unsigned to = smem_u32(sc.rows);
#pragma unroll 8
        for (int x = lane; x < C * CR; x += 32) {
            const int r = x / CR, n = (x % CR) * E;
            const bool ok = t0 + r < p.seqlen && n < p.N;
            const size_t off = ok ? size_t(r) * krow + n : 0;
            cp_async_16z(to + r * ROW + n * int(sizeof(Tin)), kp + off, ok);
            cp_async_16z(to + C * ROW + r * ROW + n * int(sizeof(Tin)), qp + off, ok);
        }
        cp_async_commit();
    }
    // lane t: a and beta of the chunk's token t
    float av = 0.f, beta = 0.f;
    if (t0 + lane < p.seqlen) {
        const size_t at = (size_t(b) * p.seqlen + t0 + lane) * p.heads + h;
        av = p.a[at];
        beta = p.beta[at];
    }
    cp_async_wait<0>();
    __syncwarp();

    // k.k and q.k in tiles [16 x 8]: rows 0-15 against tokens 0-15, rows 16-31 against all
    float kk[6][4], qk[6][4];
#pragma unroll
    for (int i = 0; i < 6; ++i) { zero4(kk[i]); zero4(qk[i]); }
    // largest |k| of the lane in rows g, g + 8, g + 16, g + 24, and |q| (bits; bf16: packed pairs)
    unsigned bigk[4] = {0, 0, 0, 0}, bigq = 0;
#pragma unroll
    for (int j = 0; j < NP / 16; ++j) {
        unsigned ka[2][KP][4], qa[2][KP][4];                    // A operands of rows 0-15 and 16-31
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if constexpr (KP == 1) {
                const unsigned at = smem_u32(sc.rows) + (16 * m + (lane & 15)) * ROW + (lane >> 4) * 16 + j * 32;
                ldsm4(ka[m][0], at);
                ldsm4(qa[m][0], at + C * ROW);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    bigk[2 * m + (y & 1)] = __vmaxu2(bigk[2 * m + (y & 1)], ka[m][0][y] & 0x7fff7fffu);
                    bigq = __vmaxu2(bigq, qa[m][0][y] & 0x7fff7fffu);
                }
            } else {
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const float2 f = *reinterpret_cast<const float2 *>(sc.rows[z] + (16 * m + g + 8 * (y & 1)) * ROW +
                                                                           (16 * j + 8 * (y >> 1) + 2 * t4) * 4);
                        unsigned x[3];
                        split_bf16(f.x, f.y, x);
#pragma unroll
                        for (int i = 0; i < 3; ++i) (z ? qa : ka)[m][i][y] = x[i];
                        unsigned &big = z ? bigq : bigk[2 * m + (y & 1)];
                        big = max(big, max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))));
                    }
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            unsigned kb[KP][4];
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                kb[i][0] = ka[n][i][0]; kb[i][1] = ka[n][i][2]; kb[i][2] = ka[n][i][1]; kb[i][3] = ka[n][i][3];
            }
#pragma unroll
            for (int m = n; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma_exact<KP>(kk[2 * (m + n) + i], ka[m], kb, i);
                    mma_exact<KP>(qk[2 * (m + n) + i], qa[m], kb, i);
                }
        }
    }
    auto whole = [](unsigned b) { return KP == 1 ? max(b << 16, b & 0xffff0000u) : b; };
    const Pow2 cq = pow2_for(__reduce_max_sync(0xffffffffu, whole(bigq)));
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        unsigned b = whole(bigk[m]);
        b = max(b, __shfl_xor_sync(0xffffffffu, b, 1));
        b = max(b, __shfl_xor_sync(0xffffffffu, b, 2));
        if (t4 == 0) sc.ck[8 * m + g] = pow2_for(b).c;
    }
    __syncwarp();
    const float ck = sc.ck[lane], ick = 1.f / ck, len = ick * 8192.f;      // of token `lane` (powers of two: exact)
    if (h == hk * group) {          // the rows as operands
        unsigned char *out = p.rows + ((size_t(b) * p.qk_heads + hk) * nchunk + c) * Rows::BYTES;
        constexpr int CR = NP / 8;
#pragma unroll 4
        for (int x = lane; x < C * CR; x += 32) {
            const int r = x / CR, n = (x % CR) * 8;
            const float cr = sc.ck[r];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float f[8];
                load8<Tin>(reinterpret_cast<const Tin *>(sc.rows[m] + r * ROW) + n, f);
                unsigned w[4][OP];
#pragma unroll
                for (int y = 0; y < 4; ++y) split_f16<OP>(f2(f[2 * y], f[2 * y + 1]), m ? cq.c : cr, w[y]);
#pragma unroll
                for (int i = 0; i < OP; ++i)
                    *reinterpret_cast<uint4 *>(out + (m * OP + i) * Rows::PIECE + r * Rows::ROW + n * 2) =
                        make_uint4(w[0][i], w[1][i], w[2][i], w[3][i]);
            }
        }
    }
    __syncwarp();                   // the rows' memory is the scratch of what follows
    float *rat = sc.rat, *at = sc.at;
    // r(t, s): lane s + 1 adds up a from token s + 1 on (no differences of long sums, so
    // a = -inf, a full reset, is exact); lane 0 is the chunk's start
    float acc = 0.f;
#pragma unroll
    for (int t = 0; t < C; ++t) {
        const float at = __shfl_sync(0xffffffffu, av, t);
        acc = t >= lane ? acc + at : 0.f;
        rat[t * RATROW + lane] = t >= lane - 1 ? ex2_approx(acc * kLog2e) : 0.f;
    }
    rat[lane * RATROW + C] = lane == C - 1 ? 1.f : 0.f;
    __syncwarp();
    float *vec = reinterpret_cast<float *>(sc.block + Block::OFF_VEC), *one = vec + kVecScalars * C;
    {
        const float gam = rat[lane * RATROW], end = rat[(C - 1) * RATROW + lane + 1];
        vec[kVecGk * C + lane] = gam * ick;
        vec[kVecSgq * C + lane] = p.scale * gam * cq.inv;
        vec[kVecBeta * C + lane] = beta;
        vec[kVecEk * C + lane] = end * ick;
        vec[kVecEbk * C + lane] = end * beta * ick;
        vec[kVecBl * C + lane] = beta * len;
        vec[kVecL * C + lane] = len;
        sc.beta[lane] = beta * len * len;
        if (lane == 0) {
            one[kGamLast] = rat[(C - 1) * RATROW];
            one[kInvQ] = cq.inv;
        }
    }
    // A and Pm: the products times their decays, over the keys' lengths
    constexpr float kOne = 1.f / 8192.f;                        // 1 / l = ck 2^-13
    float mp = 0.f;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n <= m; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s0 = 16 * n + 8 * i + 2 * t4;
                const float l0 = sc.ck[s0] * kOne, l1 = sc.ck[s0 + 1] * kOne;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int t = 16 * m + 8 * r + g;
                    const float *ak = kk[2 * (m + n) + i] + 2 * r;
                    float *pq = qk[2 * (m + n) + i] + 2 * r;
                    const float r0 = rat[t * RATROW + s0 + 1], r1 = rat[t * RATROW + s0 + 2], lt = sc.ck[t] * kOne;
                    at[s0 * NROW + t] = s0 < t ? ak[0] * lt * l0 * r0 : 0.f;
                    at[(s0 + 1) * NROW + t] = s0 + 1 < t ? ak[1] * lt * l1 * r1 : 0.f;
                    pq[0] = s0 <= t ? pq[0] * l0 * r0 * p.scale : 0.f;
                    pq[1] = s0 + 1 <= t ? pq[1] * l1 * r1 * p.scale : 0.f;
                    mp = fmaxf(mp, fmaxf(fabsf(pq[0]), fabsf(pq[1])));
                }
            }
    const Pow2 sp = pow2_for(warp_max_bits(mp));
    if (lane == 0) one[kInvP] = sp.inv;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n <= m; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float *pq = qk[2 * (m + n) + i] + 2 * r;
                    unsigned char *to = sc.block + (m + n) * kTri + tri_at(8 * r + g, i) + t4 * 4;
                    unsigned w[2];
                    split_f16<2>(f2(pq[0], pq[1]), sp.c, w);
#pragma unroll
                    for (int y = 0; y < 2; ++y) *reinterpret_cast<unsigned *>(to + Block::OFF_P + 3 * y * kTri) = w[y];
                }
    __syncwarp();
    // G of the two diagonal tiles, G (I + diag(beta) A) = A: lane t solves its row from the
    // diagonal leftwards, G(t,s) = A(t,s) - sum_{s<r<t} G(t,r) beta_r A(r,s)
    const int blk = lane >> 4, tl = lane & 15;
    float G[16], Gb[16];                                        // G(t, .) and G(t, .) beta
    {
        const float *ab = at + 16 * blk * NROW + 16 * blk;
#pragma unroll
        for (int s = 15; s >= 0; --s) {
            float x0 = ab[s * NROW + tl], x1 = 0.f;             // 0 for s >= t
#pragma unroll
            for (int r4 = (s + 1) / 4; r4 < 4; ++r4) {
                const float4 a4 = *reinterpret_cast<const float4 *>(ab + s * NROW + 4 * r4);
                const float av[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (4 * r4 + m > s) {
                        if (m & 1) x1 = fmaf(-Gb[4 * r4 + m], av[m], x1);
                        else x0 = fmaf(-Gb[4 * r4 + m], av[m], x0);
                    }
            }
            G[s] = s < tl ? x0 + x1 : 0.f;
            Gb[s] = G[s] * sc.beta[16 * blk + s];
        }
    }
    // rows of 20: G11, then G22 beta2, then Z beta1
    float *G1 = rat, *G2 = rat + 16 * 20, *Z = rat + 2 * 16 * 20;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const float *f = blk ? Gb : G;
        *reinterpret_cast<float4 *>((blk ? G2 : G1) + tl * 20 + 4 * x) = make_float4(f[4 * x], f[4 * x + 1], f[4 * x + 2], f[4 * x + 3]);
    }
    __syncwarp();
    // G21 = Z - (Z beta1) G11, Z = A21 - (G22 beta2) A21: a lane forms 8 values of row tl, columns
    // 8 blk on
    float z[8], y[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) z[x] = at[(8 * blk + x) * NROW + 16 + tl];
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
        const float4 gr = *reinterpret_cast<const float4 *>(G2 + tl * 20 + 4 * r4);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const float4 a4 = *reinterpret_cast<const float4 *>(at + (8 * blk + x) * NROW + 16 + 4 * r4);
            z[x] = fmaf(-gr.x, a4.x, fmaf(-gr.y, a4.y, fmaf(-gr.z, a4.z, fmaf(-gr.w, a4.w, z[x]))));
        }
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) { y[x] = z[x]; z[x] *= sc.beta[8 * blk + x]; }
    *reinterpret_cast<float4 *>(Z + tl * 20 + 8 * blk) = make_float4(z[0], z[1], z[2], z[3]);
    *reinterpret_cast<float4 *>(Z + tl * 20 + 8 * blk + 4) = make_float4(z[4], z[5], z[6], z[7]);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const float t = -Z[tl * 20 + r];
        const float4 lo = *reinterpret_cast<const float4 *>(G1 + r * 20 + 8 * blk);
        const float4 hi = *reinterpret_cast<const float4 *>(G1 + r * 20 + 8 * blk + 4);
        y[0] = fmaf(t, lo.x, y[0]); y[1] = fmaf(t, lo.y, y[1]); y[2] = fmaf(t, lo.z, y[2]); y[3] = fmaf(t, lo.w, y[3]);
        y[4] = fmaf(t, hi.x, y[4]); y[5] = fmaf(t, hi.y, y[5]); y[6] = fmaf(t, hi.z, y[6]); y[7] = fmaf(t, hi.w, y[7]);
    }
    float mt = 0.f;
#pragma unroll
    for (int x = 0; x < 16; ++x) mt = fmaxf(mt, fmaxf(fabsf(G[x]), fabsf(y[x & 7])));
    const Pow2 st = pow2_for(warp_max_bits(mt));
    if (lane == 0) one[kInvG] = st.inv;
    auto put = [&](int tile, int row, int half, const float *f) {     // 8 values of a row of G's tile
        unsigned x[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_f16<2>(f2(f[2 * i], f[2 * i + 1]), st.c, x[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4 *>(sc.block + (3 * i + tile) * kTri + tri_at(row, half)) =
                make_uint4(x[0][i], x[1][i], x[2][i], x[3][i]);
    };
    put(2 * blk, tl, 0, G);
    put(2 * blk, tl, 1, G + 8);
    put(1, tl, blk, y);
    // the block to global memory, one bulk copy
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        unsigned char *out = p.prep + ((size_t(b) * p.heads + h) * nchunk + c) * Block::BYTES;
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(out), "r"(smem_u32(sc.block)),
                     "r"(int(Block::BYTES)) : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
}

// Addresses of a 16 x 16 tile's B operand (n-tiles 0, 1) for ldmatrix: rows are n (plain
// load) or k (transposing load).
__device__ __forceinline__ unsigned b_rows_n(int lane, int rowbytes) {
    return unsigned(((lane >> 4) * 8 + (lane & 7)) * rowbytes + (lane >> 3 & 1) * 16);
}
__device__ __forceinline__ unsigned b_rows_k(int lane, int rowbytes) {
    return unsigned(((lane >> 3 & 1) * 8 + (lane & 7)) * rowbytes + (lane >> 4) * 16);
}
__device__ __forceinline__ unsigned tri_rows_n(int lane) { return tri_at((lane >> 4) * 8 + (lane & 7), lane >> 3 & 1); }
__device__ __forceinline__ unsigned tri_rows_k(int lane) { return tri_at((lane >> 3 & 1) * 8 + (lane & 7), lane >> 4); }

// A warp's [16 rows x 32 tokens] in accumulator layout: four tiles of 8 tokens.
using Tok = float[4][4];

// From staged rows [token][row].
template <typename T>
__device__ __forceinline__ void load_tok(const unsigned char *row0, int rowbytes, int lane, Tok &v) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unsigned r[4];
            ldsm4_t(r, smem_u32(row0) + 16 * h * rowbytes + b_rows_k(lane, rowbytes));
#pragma unroll
            for (int m = 0; m < 4; ++m) {      // m & 1: token half, m >> 1: row half
                const float2 f = bf16x2_to_f2(r[m]);
                v[2 * h + (m & 1)][2 * (m >> 1)] = f.x;
                v[2 * h + (m & 1)][2 * (m >> 1) + 1] = f.y;
            }
        }
    } else {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                v[n][x] = *reinterpret_cast<const float *>(row0 + (8 * n + 2 * t4 + (x & 1)) * rowbytes +
                                                           (g + 8 * (x >> 1)) * 4);
    }
}

// To out[token][row] rows of `stride` values, bf16 through the warp's shared tile (16-byte
// stores), fp32 straight (8 lanes cover 32 bytes).
template <typename T>
__device__ __forceinline__ void store_tok(T *out, size_t stride, int ntok, int nrow, unsigned char *tile, int lane,
                                          const Tok &o) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unsigned r[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float *c = o[2 * h + (m & 1)];
                r[m] = pack_bf16x2(c[2 * (m >> 1)], c[2 * (m >> 1) + 1]);
            }
            stsm4_t(smem_u32(tile) + b_rows_k(lane, kOutRow), r);
            __syncwarp();
            const int tok = 16 * h + (lane >> 1), half = lane & 1;
            const uint4 w = *reinterpret_cast<const uint4 *>(tile + (lane >> 1) * kOutRow + half * 16);
            if (tok < ntok && half * 8 < nrow) *reinterpret_cast<uint4 *>(out + size_t(tok) * stride + half * 8) = w;
            __syncwarp();
        }
    } else {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int tok = 8 * n + 2 * t4 + (x & 1), row = g + 8 * (x >> 1);
                if (tok < ntok && row < nrow) out[size_t(tok) * stride + row] = o[n][x];
            }
    }
}

// The scales of a lane's two rows, g and g + 8: of values whose largest magnitudes in the lane are
// m0 and m1 (the four lanes of a row join theirs).
struct RowScale {
    Pow2 r[2];
    __device__ __forceinline__ void set(float m0, float m1) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        r[0] = pow2_for(__float_as_uint(m0));
        r[1] = pow2_for(__float_as_uint(m1));
    }
    __device__ __forceinline__ float inv(int m) const { return r[m >> 1].inv; }      // of accumulator value m
};

// The largest magnitudes of a Tok in a lane's rows g and g + 8.
__device__ __forceinline__ float2 max_rows(const Tok &x) {
    float2 m = f2(0.f, 0.f);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        m.x = fmaxf(m.x, fmaxf(fabsf(x[n][0]), fabsf(x[n][1])));
        m.y = fmaxf(m.y, fmaxf(fabsf(x[n][2]), fabsf(x[n][3])));
    }
    return m;
}
__device__ __forceinline__ RowScale scale_of(const Tok &x) {
    const float2 m = max_rows(x);
    RowScale c;
    c.set(m.x, m.y);
    return c;
}
__device__ __forceinline__ unsigned max_tok(const Tok &x) {        // over the warp, as bits
    const float2 m = max_rows(x);
    return warp_max_bits(fmaxf(m.x, m.y));
}

// A Tok times its rows' scales as the pieces of two A operands (tokens 0-15 and 16-31 as the inner
// index).
template <int NP> __device__ __forceinline__ void split_tok(const Tok &x, const RowScale &c, unsigned (&a)[2][NP][4]) {
    split_tiles<NP>(x[0], x[1], c.r[0].c, c.r[1].c, a[0]);
    split_tiles<NP>(x[2], x[3], c.r[0].c, c.r[1].c, a[1]);
}

// d += x M^T (d[., t] = sum_s x[., s] M(t, s)), or with REV x M, for a lower triangle M at
// `at` in PB pieces; x in PA pieces.
template <int PA, int PB, bool REV>
__device__ __forceinline__ void mma_triangle(Tok &d, const unsigned (&x)[2][PA][4], unsigned at) {
#pragma unroll
    for (int bt = 0; bt < 2; ++bt)
#pragma unroll
        for (int bs = 0; bs <= bt; ++bs) {
            constexpr int P = PB;
            unsigned m[P][4];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if constexpr (REV) ldsm4_t(m[i], at + (3 * i + bt + bs) * kTri);
                else ldsm4(m[i], at + (3 * i + bt + bs) * kTri);
            }
            const int out = REV ? bs : bt, in = REV ? bt : bs;
#pragma unroll
            for (int n = 0; n < 2; ++n) mma_pieces<PA, PB>(d[2 * out + n], x[in], m, n);
        }
}

__device__ __forceinline__ void zero_tok(Tok &x) {
#pragma unroll
    for (int n = 0; n < 4; ++n) zero4(x[n]);
}

// x[., t] times f[t], a vector over the chunk's tokens in shared memory.
__device__ __forceinline__ void scale_tok(Tok &out, const Tok &x, const float *f, int t4) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const float2 w = *reinterpret_cast<const float2 *>(f + 8 * n + 2 * t4);
        out[n][0] = w.x * x[n][0]; out[n][1] = w.y * x[n][1];
        out[n][2] = w.x * x[n][2]; out[n][3] = w.y * x[n][3];
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT, Cfg::CTAS) delta_chain_kernel(const DeltaArgs p) {
    using Tv = typename Cfg::Tv;
    using Tout = typename Cfg::Tout;
    using Block = typename Cfg::Block;
    constexpr int C = Cfg::C, NP = Cfg::NP, NW = Cfg::NW, MODE = Cfg::MODE, KP = Cfg::KP, PV = Cfg::PV;
    constexpr bool REV = MODE == 2 || MODE == 4, BWD = Cfg::BWD, STATE = MODE == 3 || MODE == 4, MAP = MODE == 3;
    constexpr bool OUT = MODE == 0;                        // y as well
    extern __shared__ __align__(128) unsigned char delta_smem[];
    unsigned char *smem = delta_smem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // MAP: after the slices of headdim come those of the identity's rows (dstate of them)
    const int nslice = MAP ? p.slices + (p.N + 16 * NW - 1) / (16 * NW) : p.slices;
    const int slice0 = int(blockIdx.x % unsigned(nslice)), bh = int(blockIdx.x / unsigned(nslice));
    const bool ident = MAP && slice0 >= p.slices;
    const int slice = ident ? slice0 - p.slices : slice0, rows = ident ? p.N : p.P;
    const int seg = int(blockIdx.y);
    // the first segment starts from h0 itself; nothing starts from the last one's end (reverse
    // passes: from the other end)
    const int nseg = int(gridDim.y);
    const bool inner = REV ? seg + 1 < nseg : seg > 0;     // not the segment that starts from h0
    if (STATE && (seg == (REV ? 0 : nseg - 1) || (ident && seg == 0))) return;
    const int b = bh / p.heads, h = bh - b * p.heads;
    const int nchunk = (p.seqlen + C - 1) / C;
    // this segment's steps; chunk of loop step i: forwards, or backwards in the reverse pass
    const int first = seg * p.seg_chunks, count = min(p.seg_chunks, nchunk - first);
    auto chunk_of = [&](int i) { return REV ? first + count - 1 - i : first + i; };

    const int hk = h / (p.heads / p.qk_heads), prow = rows - slice * NW * 16;
    const size_t vrow = size_t(p.heads) * p.P;
    const int active = min(NW, (prow + 15) / 16);          // warps with rows
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR), *empty = full + Cfg::STAGES;
    if (tid == 0) {
        for (int i = 0; i < Cfg::STAGES; ++i) {
            mbar_init(&full[i], 1 + 32);                   // the bulk copies, a warp of cp.async
            mbar_init(&empty[i], active);
        }
        mbar_fence_init();
    }
    __syncthreads();
    // a bounded wait; after one that gave up the results are void and nothing waits any more
    bool alive = true;
    auto wait = [&](uint64_t *bar, int parity) {
        if (!mbar_test(bar, uint32_t(parity) & 1) && alive && !mbar_wait(bar, uint32_t(parity) & 1, kDeltaWaitCycles)) {
            alive = false;
            atomicAdd(p.timeouts, 1u);
        }
    };

    // Start the copies of loop step i into its stage, once the warps are done with what is there:
    // lane 0 the operands and the block, all lanes the rows of v, zeros past the end and past
    // headdim.
    const size_t voff = size_t(b) * p.seqlen * vrow + size_t(h) * p.P + slice * NW * 16;
    auto copy_v = [&](unsigned dst, int rowbytes, const auto *src, int ntok) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
        constexpr int E = 16 / sizeof(T), CR = NW * 16 / E, STEP = 32 / CR;          // copies per row, rows per round
        const int r0 = lane / CR, n = (lane % CR) * E, rows = n < prow ? ntok - r0 : 0;
        const T *at = src + r0 * vrow + n;
        dst += r0 * rowbytes + n * int(sizeof(T));
#pragma unroll
        for (int i = 0; i < C / STEP; ++i) {
            cp_async_16z(dst + i * STEP * rowbytes, i * STEP < rows ? at : src, i * STEP < rows);
            at += STEP * vrow;
        }
    };
    auto issue = [&](int i) {
        const int c = chunk_of(i), ntok = min(C, p.seqlen - c * C), slot = i % Cfg::STAGES;
        unsigned char *st = smem + slot * Cfg::STAGE;
        if (i >= Cfg::STAGES) wait(&empty[slot], i / Cfg::STAGES - 1);
        if (lane == 0) {
            mbar_arrive_expect_tx(&full[slot], Cfg::Rows::BYTES + Block::BYTES);
            bulk_load(st, p.rows + ((size_t(b) * p.qk_heads + hk) * nchunk + c) * Cfg::Rows::BYTES, Cfg::Rows::BYTES,
                      &full[slot]);
            bulk_load(st + Cfg::OFF_TRI, p.prep + (size_t(bh) * nchunk + c) * Block::BYTES, Block::BYTES, &full[slot]);
        }
        __syncwarp();
        const size_t at = voff + size_t(c) * C * vrow;
        if (!ident) copy_v(smem_u32(st) + Cfg::OFF_V, Cfg::VROW, static_cast<const Tv *>(p.v) + at, ntok);
        mbar_arrive_cp_async(&full[slot]);
    };
    if (warp == 0)
        for (int i = 0; i + 1 < Cfg::STAGES && i < count; ++i) issue(i);

    const int g = lane >> 2, t4 = lane & 3;
    const int p0 = slice * NW * 16 + warp * 16;           // the warp's first row
    const int nrow = rows - p0;                            // its rows (<= 0: none, may exceed 16)
    float s[NP / 8][4];
    const size_t sbase = size_t(bh) * p.P * p.N;
    auto state_io = [&](auto f) {                          // f(accumulator pair, offset) of each pair held
#pragma unroll
        for (int j = 0; j < NP / 8; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = g + 8 * r, col = 8 * j + 2 * t4;
                if (row < nrow && col < p.N) f(s[j][2 * r], s[j][2 * r + 1], size_t(p0 + row) * p.N + col);
            }
    };
#pragma unroll
    for (int j = 0; j < NP / 8; ++j) zero4(s[j]);
    const float *start = ident || (STATE && inner) ? nullptr
                         : inner ? p.seg_state + (size_t(bh) * nseg + (REV ? seg + 1 : seg - 1)) * p.P * p.N
                         : p.h0 ? p.h0 + sbase : nullptr;
    if (start != nullptr)
        state_io([&](float &x, float &y, size_t off) {
            const float2 f = *reinterpret_cast<const float2 *>(start + off);
            x = f.x; y = f.y;
        });
    if (ident) {                                           // rows of the identity, and no v
#pragma unroll
        for (int j = 0; j < NP / 8; ++j)
#pragma unroll
            for (int m = 0; m < 4; ++m) s[j][m] = p0 + g + 8 * (m >> 1) == 8 * j + 2 * t4 + (m & 1) ? 1.f : 0.f;
        for (int i = 0; i < Cfg::STAGES; ++i)              // each warp its own columns of the staged rows
            for (int x = lane; x < C * sizeof(Tv); x += 32)
                *reinterpret_cast<uint4 *>(smem + i * Cfg::STAGE + Cfg::OFF_V + (x / sizeof(Tv)) * Cfg::VROW +
                                           warp * 16 * sizeof(Tv) + (x % sizeof(Tv)) * 16) = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }
    unsigned char *tile = smem + Cfg::OFF_OUT + warp * Cfg::OUT;
    const unsigned bn = b_rows_n(lane, Cfg::KROW), bk = b_rows_k(lane, Cfg::KROW);
    const unsigned tr = REV ? tri_rows_k(lane) : tri_rows_n(lane);
    const int nbound = (p.seqlen + kDeltaSave - 1) / kDeltaSave + 1;       // boundaries, the end among them
    const size_t part = slice * NW + warp, parts = size_t(p.slices) * NW;
    // a shared tile to global memory, as it stands
    auto copy_out = [&](unsigned char *to, const unsigned char *from, auto bytes) {
        __syncwarp();
#pragma unroll
        for (int x = 0; x < decltype(bytes)::value / 512; ++x)
            *reinterpret_cast<uint4 *>(to + 512 * x + 16 * lane) = *reinterpret_cast<const uint4 *>(from + 512 * x + 16 * lane);
        __syncwarp();
    };
    const int srow = (lane >> 3 & 1) * 8 + (lane & 7), spiece = lane >> 4;       // stmatrix: row and piece of the lane
    // a Tok times c as the last kernel reads it, in `pieces` pieces
    auto keep_tok16 = [&](auto pieces, unsigned char *to, const Tok &f, float k, int c) {
        constexpr int NPC = decltype(pieces)::value;
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
            unsigned r[NPC][4];
            split_tiles<NPC>(f[2 * h2], f[2 * h2 + 1], k, r);
#pragma unroll
            for (int i = 0; i < NPC; ++i) stsm4(smem_u32(tile) + i * kTok16 + tok16_at(srow, 2 * h2 + spiece), r[i]);
        }
        copy_out(to + ((size_t(bh) * nchunk + c) * parts + part) * (NPC * kTok16), tile, std::integral_constant<int, NPC * kTok16>());
    };
    // the state times c, in two pieces
    auto keep_state16 = [&](unsigned char *to, float k, int x) {
#pragma unroll
        for (int n = 0; n < NP / 32; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                unsigned A[2][4];
                split_tiles<2>(s[4 * n + 2 * j], s[4 * n + 2 * j + 1], k, A);
#pragma unroll
                for (int i = 0; i < 2; ++i) stsm4(smem_u32(tile) + i * kTok16 + tok16_at(srow, 2 * j + spiece), A[i]);
            }
            copy_out(to + (((size_t(bh) * nbound + x) * (NP / 32) + n) * parts + part) * (2 * kTok16), tile,
                     std::integral_constant<int, 2 * kTok16>());
        }
    };
    using std::integral_constant;
    if (nrow <= 0) return;                                 // rows past headdim
    int turn = warp + 1;                                   // loop steps until it is this warp's to start copies
    // the largest magnitudes of the lane's two rows of the state, kept up with its updates
    float ms[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NP / 8; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) ms[m >> 1] = fmaxf(ms[m >> 1], fabsf(s[j][m]));

    for (int i = 0; i < count; ++i) {
        const int c = chunk_of(i);
        constexpr int CS = kDeltaSave / C;
        const size_t tok0 = (size_t(b) * p.seqlen + size_t(c) * C) * p.heads + h;
        const int ntok = min(C, p.seqlen - c * C);
        RowScale cS;
        cS.set(ms[0], ms[1]);
        if constexpr (MODE == 1)
            if (c % CS == 0) {
                const unsigned msb = warp_max_bits(fmaxf(ms[0], ms[1]));
                keep_state16(p.s16, pow2_for(msb).c, c / CS);
                if (lane == 0) p.smax[(size_t(bh) * nbound + c / CS) * parts + part] = msb;
            }
        if constexpr (MODE == 2)
            if (c % CS == CS - 1 || c == nchunk - 1) {
                const unsigned msb = warp_max_bits(fmaxf(ms[0], ms[1]));
                keep_state16(p.d16, pow2_for(msb).c, c / CS + 1);
                if (lane == 0) p.smax[(size_t(bh) * nbound + c / CS + 1) * parts + part] = msb;
            }

        const int slot = i % Cfg::STAGES;
        wait(&full[slot], i / Cfg::STAGES);
        const unsigned char *stage = smem + slot * Cfg::STAGE;
        const float *vec = reinterpret_cast<const float *>(stage + Cfg::OFF_TRI + Block::OFF_VEC);
        const unsigned kbase = smem_u32(stage + Cfg::OFF_K), qbase = smem_u32(stage + Cfg::OFF_Q);
        const unsigned tbase = smem_u32(stage + Cfg::OFF_TRI) + tr;
        const float *one = vec + kVecScalars * C;
        // S k, and S q for y; the next step's operands are loaded ahead of this one's products
        Tok sk, sq;
        zero_tok(sk); zero_tok(sq);
        unsigned kb[2][KP][4], qb[2][KP][4];
        auto load_kq = [&](int j) {
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                for (int m = 0; m < KP; ++m) {
                    ldsm4(kb[h2][m], kbase + m * Cfg::PIECE + 16 * h2 * Cfg::KROW + bn + j * 32);
                    if constexpr (OUT) ldsm4(qb[h2][m], qbase + m * Cfg::PIECE + 16 * h2 * Cfg::KROW + bn + j * 32);
                }
        };
        load_kq(0);
#pragma unroll
        for (int j = 0; j < NP / 16; ++j) {
            unsigned A[2][4];
            split_tiles<2>(s[2 * j], s[2 * j + 1], cS.r[0].c, cS.r[1].c, A);
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma_pieces<2, KP>(sk[2 * h2 + n], A, kb[h2], n);
                    if constexpr (OUT) mma_pieces<2, KP>(sq[2 * h2 + n], A, qb[h2], n);
                }
            if (j + 1 < NP / 16) load_kq(j + 1);
        }
        // By now the other warps have left the stage that comes next (or soon will): the one whose
        // turn it is starts the copies into it.
        if (--turn == 0) {
            turn = active;
            if (i + Cfg::STAGES - 1 < count) issue(i + Cfg::STAGES - 1);
        }
        Tok v, x, du;
        load_tok<Tv>(stage + Cfg::OFF_V + warp * 16 * int(sizeof(Tv)), Cfg::VROW, lane, v);
        unsigned mv = 0;                                   // reverse pass: largest |dO|
        (void)mv;
        if constexpr (!REV) {
            // R = v - gam S k
            scale_tok(sk, sk, vec + kVecGk * C, t4);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) x[n][m] = fmaf(-cS.inv(m), sk[n][m], v[n][m]);
        } else {
            // rhs = end (dS k) + Pm^T dO, times beta
            Tok lo;
            unsigned A[2][PV][4];
            const RowScale cv = scale_of(v);
            if constexpr (MODE == 2) mv = max_tok(v);
            split_tok<PV>(v, cv, A);
            zero_tok(lo);
            mma_triangle<PV, 2, true>(lo, A, tbase + Block::OFF_P);
            scale_tok(lo, lo, vec + kVecL * C, t4);
            scale_tok(sk, sk, vec + kVecEk * C, t4);
            const float f[2] = {one[kInvP] * cv.r[0].inv, one[kInvP] * cv.r[1].inv};
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) du[n][m] = fmaf(cS.inv(m), sk[n][m], f[m >> 1] * lo[n][m]);
        }
        // e = R - G (beta R), or du = rhs - G^T (beta rhs) and w = beta du.  Every operand's scale
        // comes from its own largest value.
        {
            unsigned A[2][2][4];
            Tok d;
            scale_tok(d, REV ? du : x, vec + kVecBl * C, t4);
            const RowScale cx = scale_of(d);
            split_tok<2>(d, cx, A);
            zero_tok(d);
            mma_triangle<2, 2, REV>(d, A, tbase);
            scale_tok(d, d, vec + kVecL * C, t4);
            const float f[2] = {-one[kInvG] * cx.r[0].inv, -one[kInvG] * cx.r[1].inv};
            Tok &to = REV ? du : x;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) to[n][m] = fmaf(f[m >> 1], d[n][m], to[n][m]);
            if constexpr (REV) scale_tok(x, du, vec + kVecBeta * C, t4);
        }
        unsigned mx = 0;                                   // backward: largest |e|, or |w|
        (void)mx;
        if constexpr (BWD) {
            mx = max_tok(x);
            if (lane == 0) {
                p.emax[(size_t(bh) * nchunk + c) * parts + part] = mx;
                if constexpr (REV) p.ymax[(size_t(bh) * nchunk + c) * parts + part] = mv;
            }
        }
        Tok o;
        if constexpr (OUT) {
            // y = scale gam S q + Pm (beta e)
            unsigned A[2][2][4];
            scale_tok(o, x, vec + kVecBl * C, t4);
            const RowScale cu = scale_of(o);
            split_tok<2>(o, cu, A);
            zero_tok(o);
            mma_triangle<2, 2, false>(o, A, tbase + Block::OFF_P);
            scale_tok(sq, sq, vec + kVecSgq * C, t4);
            const float f[2] = {one[kInvP] * cu.r[0].inv, one[kInvP] * cu.r[1].inv};
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) o[n][m] = fmaf(f[m >> 1], o[n][m], cS.inv(m) * sq[n][m]);
        }
        if constexpr (MODE == 1) {
            keep_tok16(integral_constant<int, 2>(), p.e16, x, pow2_for(mx).c, c);
        } else if constexpr (MODE == 2) {
            keep_tok16(integral_constant<int, 2>(), p.w16, x, pow2_for(mx).c, c);
            keep_tok16(integral_constant<int, PV>(), p.y16, v, pow2_for(mv).c, c);
            store_tok<Tout>(static_cast<Tout *>(p.y) + tok0 * p.P + p0, vrow, ntok, nrow, tile, lane, x);
        }
        // the state's update: operand A1 against k (and in the reverse pass A2 against q)
        const float glast = one[kGamLast];
        {
            unsigned A1[2][2][4], A2[2][REV ? 2 : 1][4];
            Tok w;
            scale_tok(w, x, vec + (REV ? kVecGk : kVecEbk) * C, t4);
            const RowScale c1 = scale_of(w);
            split_tok<2>(w, c1, A1);
            RowScale c2{};
            if constexpr (REV) {
                scale_tok(w, v, vec + kVecSgq * C, t4);
                c2 = scale_of(w);
                split_tok<2>(w, c2, A2);
            }
            auto load_t = [&](unsigned (&f)[KP][4], unsigned base, int h2, int j) {
#pragma unroll
                for (int m = 0; m < KP; ++m) ldsm4_t(f[m], base + m * Cfg::PIECE + 16 * h2 * Cfg::KROW + bk + j * 32);
            };
            const float2 gl = f2(glast, glast);
            ms[0] = ms[1] = 0.f;
#pragma unroll
            for (int j = 0; j < NP / 16; ++j) {
                float d[2][4], d2[2][4];
                zero4(d[0]); zero4(d[1]); zero4(d2[0]); zero4(d2[1]);
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    unsigned f[KP][4];
                    load_t(f, kbase, h2, j);
#pragma unroll
                    for (int n = 0; n < 2; ++n) mma_pieces<2, KP>(d[n], A1[h2], f, n);
                    if constexpr (REV) {
                        load_t(f, qbase, h2, j);
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_pieces<2, KP>(d2[n], A2[h2], f, n);
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int m = 0; m < 4; m += 2) {
                        float *at = s[2 * j + n] + m;
                        float2 u = fmul2(gl, f2(at[0], at[1]));
                        const float f1 = REV ? -c1.inv(m) : c1.inv(m);
                        if constexpr (REV) u = ffma2(f2(c2.inv(m), c2.inv(m)), f2(d2[n][m], d2[n][m + 1]), u);
                        u = ffma2(f2(f1, f1), f2(d[n][m], d[n][m + 1]), u);
                        at[0] = u.x; at[1] = u.y;
                        ms[m >> 1] = fmaxf(ms[m >> 1], fmaxf(fabsf(u.x), fabsf(u.y)));
                    }
            }
        }
        if constexpr (MODE == 0)
            store_tok<Tout>(static_cast<Tout *>(p.y) + tok0 * p.P + p0, vrow, ntok, nrow, tile, lane, o);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);         // the stage may be filled again
    }
    if (!alive)                                            // copies may still be on their way: wait (bounded) for them
        for (int i = max(0, count - Cfg::STAGES); i < count; ++i)
            mbar_wait(&full[i % Cfg::STAGES], uint32_t(i / Cfg::STAGES) & 1, kDeltaWaitCycles);
    float *end = ident ? p.seg_map + (size_t(bh) * nseg + seg) * p.N * p.N
                 : STATE ? p.seg_state + (size_t(bh) * nseg + seg) * p.P * p.N
                 : !p.hN || seg != (REV ? 0 : nseg - 1) ? nullptr
                 : p.end_slot ? p.seg_state + (size_t(bh) * nseg + seg) * p.P * p.N : p.hN + sbase;
    if (end != nullptr)
        state_io([&](float &x, float &y, size_t off) { *reinterpret_cast<float2 *>(end + off) = make_float2(x, y); });
}

// The segments' start states: behind segment 0 the state that it ended with, then
//     start(i + 1) = start(i) map(i) + end(i)
// in place of end(i); reverse passes from the last segment down, with map(i) transposed.  A CTA
// takes R rows of one head through the segments, thread j column j.
template <int R, bool REV>
__global__ void __launch_bounds__(128) delta_fold_kernel(const DeltaArgs p, int nseg) {
    __shared__ __align__(16) float row[R][128];
    const int tiles = (p.P + R - 1) / R, bh = int(blockIdx.x) / tiles, r0 = (int(blockIdx.x) % tiles) * R, j = threadIdx.x;
    const int nr = min(R, p.P - r0);
    float *st = p.seg_state + (size_t(bh) * nseg * p.P + r0) * p.N;
    const float *map = p.seg_map + size_t(bh) * nseg * p.N * p.N;
    float x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = r < nr && j < p.N ? st[(REV ? size_t(nseg - 1) * p.P * p.N : 0) + size_t(r) * p.N + j] : 0.f;
    for (int step = 1; step + 1 < nseg; ++step) {
        const int i = REV ? nseg - 1 - step : step;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) row[r][j] = x[r];
        __syncthreads();
        float *end = st + size_t(i) * p.P * p.N;
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = r < nr && j < p.N ? end[size_t(r) * p.N + j] : 0.f;
        if (j < p.N) {
            const float *m = map + size_t(i) * p.N * p.N + (REV ? size_t(j) * p.N : size_t(j));
            for (int n0 = 0; n0 < p.N; n0 += 32) {         // 32 loads on their way at once
                float f[32];
#pragma unroll
                for (int n = 0; n < 32; ++n) f[n] = n0 + n < p.N ? __ldg(m + size_t(n0 + n) * (REV ? 1 : p.N)) : 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int n = 0; n < 32; n += 4) {
                        const float4 u = *reinterpret_cast<const float4 *>(&row[r][n0 + n]);
                        x[r] = fmaf(u.x, f[n], fmaf(u.y, f[n + 1], fmaf(u.z, f[n + 2], fmaf(u.w, f[n + 3], x[r]))));
                    }
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r < nr) end[size_t(r) * p.N + j] = x[r];
        }
    }
}

}  // namespace ssm
