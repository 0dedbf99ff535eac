// delta_rule.cuh -- the gated delta rule by chunks of 16 tokens, the state in registers.
//
// Per sequence and head, with the headdim x dstate fp32 state S (dv = headdim rows, dk =
// dstate columns):
//     S' = exp(a_t) S,  e_t = v_t - S' k_t,  S = S' + beta_t e_t k_t^T,  y_t = scale S q_t
// Over a chunk of C tokens with start state S, r(t,s) = exp(a_{s+1} + ... + a_t),
// gam_t = r(t, before the chunk), end_s = r(last, s):
//     R_t = v_t - gam_t S k_t
//     e   = T R,           T = (I + n)^-1,  n(t,s) = r(t,s) (k_t.k_s) beta_s   for s < t
//     y_t = scale gam_t S q_t + sum_{s<=t} Pm(t,s) beta_s e_s,  Pm(t,s) = scale r(t,s) (q_t.k_s)
//     S  <- gam_last S + sum_s (end_s beta_s e_s) k_s^T
// Every row of S (one value of headdim) goes through this on its own, given k, q, T and Pm,
// so a warp owns 16 rows and keeps them in registers as accumulator tiles [16 x dstate]:
// the state enters each product as a register operand and no step of the chain goes through
// shared memory or waits for another warp.  What depends on k, q, a and beta alone (T, Pm and
// the decays) is formed for all chunks in parallel by delta_prep_kernel, one warp per chunk,
// and read back by the chains with the chunk's rows (cp.async, three chunks ahead).  Formed
// by an extra warp inside each chain's CTA instead it took 5100 cycles a chunk against the
// chain's own 2800 and set the pace.
//
// Precision: the products run on the tensor cores in bf16 with fp32 accumulation.  q, k, v
// in bf16 are exact operands; an fp32 operand goes in as bf16 pieces whose sum it is (three
// pieces hold all its bits, two hold 17).  Three pieces wherever the state or the
// corrections depend on it; two for T - I against R (the small part of e = R + (T - I) R)
// and for a bf16 y.  Sums into the state are fp32 additions outside the tensor core, which
// cuts off instead of rounding.
//
// Why 16 tokens: the products between tokens grow with the chunk while those with the state
// do not, and the inverse of a 16 x 16 triangle is short enough to hide in one warp.
#pragma once

#include <type_traits>

#include "mma_common.cuh"

namespace ssm {

struct DeltaArgs {
    const void *q, *k;      // [batch][seqlen][qk_heads][dstate]; the chains: bf16, or the pieces
                            // that the prep kernel made of fp32 ones, `piece` values apart
    size_t piece;
    unsigned char *prep;    // [batch][heads][chunks] blocks of the prep kernel
    __nv_bfloat16 *qp, *kp; // prep kernel: where the pieces of fp32 q, k go
    const void *v;          // [batch][seqlen][heads][headdim]; the reverse pass: dy
    const void *v2;         // backward: dy, and v in the reverse pass
    const float *a, *beta;  // [batch][seqlen][heads]
    void *y;                // forward: y; reverse pass: dv
    const float *h0;        // start state (reverse pass: the final state's gradient) or NULL
    float *hN;              // end state (reverse pass: the start state's gradient) or NULL
    float *e;               // backward: [batch][seqlen][heads][headdim], e written, then read
    float *w;               // reverse pass: the same of w, or NULL (w is then dv itself)
    float *ck;              // backward: the state at every boundary of 64 tokens and at the end,
                            // [batch][heads][boundaries][headdim][dstate]
    float *dck;             // reverse pass: its gradient there
    float *sum0, *sum1;     // backward: [slices][batch][heads][seqlen] sums over a slice's rows:
                            // dy.y; in the reverse pass v.w and (gradient of beta) e.du
    float *zsum;            // reverse pass: [slices * warps][batch][heads][boundaries] <dS, S>
    int batch, seqlen, heads, qk_heads, P, N, slices;
    float scale;
};

constexpr int kDeltaC = 16;          // tokens per chunk
constexpr int kDeltaSave = 64;       // tokens between the states kept for the backward
constexpr int kTri = 512;            // bytes of a 16 x 16 bf16 tile, rows of 32
constexpr int kOutRow = 48;          // bytes per row of a warp's output tile

// Byte offset of the 16-byte half `c` of row r in such a tile: the halves change places every
// four rows, so that eight rows' halves are eight different bank groups (ldmatrix).
__device__ __forceinline__ int tri_at(int r, int c) { return r * 32 + ((c ^ (r >> 2)) & 1) * 16; }

// What the prep kernel leaves per chunk and head: T - I in two bf16 pieces, Pm in PP pieces,
// for the backward n / beta in two, then fp32 vectors over the chunk's tokens (gam, scale
// gam, beta, end, end beta) and gam of the last token.
template <int PP_, bool BWD_> struct DeltaBlock {
    static constexpr int PP = PP_;
    static constexpr bool BWD = BWD_;
    static constexpr int NTRI = 2 + PP + (BWD ? 2 : 0);
    static constexpr int OFF_VEC = NTRI * kTri, BYTES = OFF_VEC + 6 * kDeltaC * 4;
};

// NP: dstate rounded up; NW: warps with 16 rows each.  KP: bf16 pieces of q and k.  MODE 0:
// forward (y); 1: forward of the backward pass (e and the kept states); 2: the reverse pass.
template <int NP_, int NW_, int KP_, typename Tv_, typename Tv2_, typename Tout_, int MODE_> struct DeltaCfg {
    static constexpr int NP = NP_, NW = NW_, MODE = MODE_, KP = KP_;
    using Tv = Tv_;        // v, or dy in the reverse pass
    using Tv2 = Tv2_;      // the other one
    using Tout = Tout_;
    static constexpr int C = kDeltaC, NT = 32 * NW, STAGES = 4;
    static constexpr bool F32V = sizeof(Tv) == 4;
    static constexpr int PO = MODE != 0 || sizeof(Tout) == 4 ? 3 : 2;         // pieces behind y
    using Block = DeltaBlock<PO, MODE != 0>;
    static constexpr int KROW = NP * 2 + 16;                                  // padded rows (bytes)
    static constexpr int VROW = NW * 16 * int(sizeof(Tv)) + 16;
    static constexpr int V2ROW = NW * 16 * int(sizeof(Tv2)) + 16;
    static constexpr int PIECE = C * KROW;
    static constexpr int OFF_K = 0, OFF_Q = KP * PIECE, OFF_V = 2 * KP * PIECE;
    static constexpr int OFF_V2 = OFF_V + C * VROW;
    static constexpr int OFF_TRI = OFF_V2 + (MODE != 0 ? C * V2ROW : 0);
    static constexpr int STAGE = OFF_TRI + Block::BYTES;
    static constexpr int OFF_OUT = STAGES * STAGE;                            // per-warp output tiles
    static constexpr int OFF_RED = OFF_OUT + NW * C * kOutRow;                // 2 buffers of token sums
    static constexpr int NRED = MODE;                                         // sums per token
    static constexpr int REDBUF = NRED * NW * C * 4;
    static constexpr int OFF_ST = OFF_RED + 2 * REDBUF;                       // reverse pass: kept states
    static constexpr int STROW = NP * 4 + 16;
    static constexpr int SMEM_BYTES = OFF_ST + (MODE == 2 ? NW * 16 * STROW : 0);
};

// acc += A B over the piece products that matter: all of them when one side is a single
// piece, else those whose pieces' ranks sum below the smaller count.  The leading product
// goes to `big`, the others to `small` (two short chains instead of one long one).
template <int PA, int PB>
__device__ __forceinline__ void mma_pieces(float (&big)[4], float (&small)[4], const unsigned (&a)[PA][4],
                                           const unsigned (&b)[PB][4], int tile) {
    constexpr int LIM = (PA == 1 || PB == 1) ? (PA > PB ? PA : PB) : (PA < PB ? PA : PB);
#pragma unroll
    for (int i = 0; i < PA; ++i)
#pragma unroll
        for (int j = 0; j < PB; ++j)
            if (i + j < LIM) {
                if (i + j == 0) mma_bf16(big, a[i], b[j][2 * tile], b[j][2 * tile + 1]);
                else mma_bf16(small, a[i], b[j][2 * tile], b[j][2 * tile + 1]);
            }
}

// One warp per chunk and head forms the chunk's block; of fp32 q and k also their bf16 pieces
// (by the first head of each key head).
template <int NP, typename Tin, class Block>
__global__ void __launch_bounds__(256) delta_prep_kernel(const DeltaArgs p) {
    constexpr int C = kDeltaC, RATROW = 18, NROW = 20, KP = sizeof(Tin) == 4 ? 3 : 1, J = NP / 32;
    __shared__ __align__(16) float scratch[8][C * RATROW + C * NROW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int nchunk = (p.seqlen + C - 1) / C;
    const long long id = (long long)blockIdx.x * 8 + warp;      // head fastest: neighbours share q and k rows
    if (id >= (long long)p.batch * p.heads * nchunk) return;
    const int h = int(id % p.heads);
    const long long bc = id / p.heads;
    const int c = int(bc % nchunk), b = int(bc / nchunk);
    const int group = p.heads / p.qk_heads, hk = h / group, t0 = c * C;
    float *rat = scratch[warp], *nt = rat + C * RATROW;         // rat[t][s + 1] = r(t, s), nt[s][t] = n(t, s)

    // lanes 0..15: a of the chunk's token `lane`; lanes 16..31: beta of token lane - 16
    float gate = 0.f;
    if (t0 + (lane & 15) < p.seqlen)
        gate = (lane < 16 ? p.a : p.beta)[(size_t(b) * p.seqlen + t0 + (lane & 15)) * p.heads + h];

    // k.k and q.k.  The inner index may be permuted at will, so a lane takes 8 neighbouring
    // values of its rows g and g + 8: two steps' operands in one 16-byte load.
    float kk[2][4], qk[2][4], kks[2][4], qks[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) { zero4(kk[i]); zero4(qk[i]); zero4(kks[i]); zero4(qks[i]); }
    const size_t krow = size_t(p.qk_heads) * p.N;
    const size_t k0 = (size_t(b) * p.seqlen + t0) * krow + size_t(hk) * p.N;
    uint4 rows[2][2][J][KP];                                    // [k, q][row half][32 columns][piece]
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int t = g + 8 * r, n = 32 * j + 8 * t4;
                const bool ok = t0 + t < p.seqlen && n < p.N;
                const size_t off = k0 + size_t(t) * krow + n;
                const Tin *src = static_cast<const Tin *>(m ? p.q : p.k);
                uint4 (&w)[KP] = rows[m][r][j];
                if constexpr (KP == 1) {
                    w[0] = ok ? __ldg(reinterpret_cast<const uint4 *>(src + off)) : make_uint4(0, 0, 0, 0);
                } else {
                    float f[8] = {};
                    if (ok) load8<float>(src + off, f);
                    unsigned x[4][3];
#pragma unroll
                    for (int y = 0; y < 4; ++y) split_pair<3>(f[2 * y], f[2 * y + 1], x[y]);
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        w[i] = make_uint4(x[0][i], x[1][i], x[2][i], x[3][i]);
                        if (ok && h == hk * group)
                            *reinterpret_cast<uint4 *>((m ? p.qp : p.kp) + i * p.piece + off) = w[i];
                    }
                }
            }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            unsigned ka[KP][4], qa[KP][4], kb[KP][4];
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                auto half = [&](const uint4 &w, int x) { return st ? (x ? w.w : w.z) : (x ? w.y : w.x); };
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        ka[i][2 * x + r] = half(rows[0][r][j][i], x);
                        qa[i][2 * x + r] = half(rows[1][r][j][i], x);
                        kb[i][2 * r + x] = ka[i][2 * x + r];
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mma_pieces<KP, KP>(kk[i], kks[i], ka, kb, i);
                mma_pieces<KP, KP>(qk[i], qks[i], qa, kb, i);
            }
        }
    // r(t, s): lane s + 1 adds up a from token s + 1 on (no differences of long sums, so
    // a = -inf, a full reset, is exact); lane 0 is the chunk's start
    float acc = 0.f;
#pragma unroll
    for (int t = 0; t < C; ++t) {
        const float at = __shfl_sync(0xffffffffu, gate, t);
        acc = t >= lane ? acc + at : 0.f;
        if (lane <= C) rat[t * RATROW + lane] = t >= lane - 1 ? ex2_approx(acc * kLog2e) : 0.f;
    }
    __syncwarp();
    unsigned char *out = p.prep + ((size_t(b) * p.heads + h) * nchunk + c) * Block::BYTES;
    float *vec = reinterpret_cast<float *>(out + Block::OFF_VEC);
    const float beta = __shfl_sync(0xffffffffu, gate, 16 + (lane & 15));
    if (lane < C) {
        const float gam = rat[lane * RATROW], end = rat[(C - 1) * RATROW + lane + 1];
        vec[lane] = gam;
        vec[C + lane] = p.scale * gam;
        vec[2 * C + lane] = beta;
        vec[3 * C + lane] = end;
        vec[4 * C + lane] = end * beta;
        if (lane == C - 1) vec[5 * C] = gam;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s0 = 8 * i + 2 * t4;
        const float b0 = __shfl_sync(0xffffffffu, beta, s0), b1 = __shfl_sync(0xffffffffu, beta, s0 + 1);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = g + 8 * r;
            const float r0 = rat[t * RATROW + s0 + 1], r1 = rat[t * RATROW + s0 + 2];
            const float k0 = s0 < t ? (kk[i][2 * r] + kks[i][2 * r]) * r0 : 0.f;
            const float k1 = s0 + 1 < t ? (kk[i][2 * r + 1] + kks[i][2 * r + 1]) * r1 : 0.f;
            nt[s0 * NROW + t] = s0 < t ? k0 * b0 : 0.f;
            nt[(s0 + 1) * NROW + t] = s0 + 1 < t ? k1 * b1 : 0.f;
            unsigned char *at = out + tri_at(t, i) + t4 * 4;
            if constexpr (Block::BWD) {
                unsigned x[2];
                split_pair<2>(k0, k1, x);
#pragma unroll
                for (int m = 0; m < 2; ++m) *reinterpret_cast<unsigned *>(at + (2 + Block::PP + m) * kTri) = x[m];
            }
            const float q0 = s0 <= t ? (qk[i][2 * r] + qks[i][2 * r]) * r0 * p.scale : 0.f;
            const float q1 = s0 + 1 <= t ? (qk[i][2 * r + 1] + qks[i][2 * r + 1]) * r1 * p.scale : 0.f;
            unsigned w[Block::PP];
            split_pair<Block::PP>(q0, q1, w);
#pragma unroll
            for (int m = 0; m < Block::PP; ++m) *reinterpret_cast<unsigned *>(at + (2 + m) * kTri) = w[m];
        }
    }
    __syncwarp();
    // lane t solves row t of T (I + n) = I from the diagonal leftwards
    if (lane < C) {
        float T[C];
#pragma unroll
        for (int s = C - 1; s >= 0; --s) {
            float x0 = 0.f, x1 = 0.f;
#pragma unroll
            for (int r4 = (s + 1) / 4; r4 < C / 4; ++r4) {
                const float4 n4 = *reinterpret_cast<const float4 *>(nt + s * NROW + 4 * r4);
                const float nv[4] = {n4.x, n4.y, n4.z, n4.w};
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (4 * r4 + m > s) {
                        if (m & 1) x1 = fmaf(-T[4 * r4 + m], nv[m], x1);
                        else x0 = fmaf(-T[4 * r4 + m], nv[m], x0);
                    }
            }
            T[s] = s == lane ? 1.f : (s < lane ? x0 + x1 : 0.f);
        }
#pragma unroll
        for (int s = 0; s < C; ++s) T[s] = s == lane ? 0.f : T[s];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            unsigned x[4][2];
#pragma unroll
            for (int y = 0; y < 4; ++y) split_pair<2>(T[8 * half + 2 * y], T[8 * half + 2 * y + 1], x[y]);
#pragma unroll
            for (int m = 0; m < 2; ++m)
                *reinterpret_cast<uint4 *>(out + m * kTri + tri_at(lane, half)) =
                    make_uint4(x[0][m], x[1][m], x[2][m], x[3][m]);
        }
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

// One warp's [16 rows x 16 tokens] tile of staged rows [token][row] in accumulator layout.
template <typename T>
__device__ __forceinline__ void load_tok_tile(const unsigned char *row0, int rowbytes, int lane, float (&v)[2][4]) {
    if constexpr (sizeof(T) == 2) {
        unsigned r[4];
        ldsm4_t(r, smem_u32(row0) + b_rows_k(lane, rowbytes));
#pragma unroll
        for (int m = 0; m < 4; ++m) {          // m & 1: token half, m >> 1: row half
            const float2 f = bf16x2_to_f2(r[m]);
            v[m & 1][2 * (m >> 1)] = f.x;
            v[m & 1][2 * (m >> 1) + 1] = f.y;
        }
    } else {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                v[i][x] = *reinterpret_cast<const float *>(row0 + (8 * i + 2 * t4 + (x & 1)) * rowbytes +
                                                           (g + 8 * (x >> 1)) * 4);
    }
}

// Store a [16 rows x 16 tokens] tile to out[token][row] rows of `stride` values, bf16 through
// the warp's shared tile (16-byte stores), fp32 straight (8 lanes cover 32 bytes).
template <typename T>
__device__ __forceinline__ void store_tok_tile(T *out, size_t stride, int ntok, int nrow, unsigned char *tile, int lane,
                                               const float (&o)[2][4]) {
    if constexpr (sizeof(T) == 2) {
        unsigned r[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) r[m] = pack_bf16x2(o[m & 1][2 * (m >> 1)], o[m & 1][2 * (m >> 1) + 1]);
        stsm4_t(smem_u32(tile) + b_rows_k(lane, kOutRow), r);
        __syncwarp();
        const int tok = lane >> 1, half = lane & 1;
        const uint4 w = *reinterpret_cast<const uint4 *>(tile + tok * kOutRow + half * 16);
        if (tok < ntok && half * 8 < nrow) *reinterpret_cast<uint4 *>(out + size_t(tok) * stride + half * 8) = w;
        __syncwarp();
    } else {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int tok = 8 * i + 2 * t4 + (x & 1), row = g + 8 * (x >> 1);
                if (tok < ntok && row < nrow) out[size_t(tok) * stride + row] = o[i][x];
            }
    }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT) delta_chain_kernel(const DeltaArgs p) {
    using Tv = typename Cfg::Tv;
    using Tout = typename Cfg::Tout;
    constexpr int C = Cfg::C, NP = Cfg::NP, NW = Cfg::NW, MODE = Cfg::MODE, KP = Cfg::KP, PO = Cfg::PO;
    extern __shared__ __align__(128) unsigned char delta_smem[];
    unsigned char *smem = delta_smem;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slice = int(blockIdx.x % unsigned(p.slices));
    const int bh = int(blockIdx.x / unsigned(p.slices));
    const int b = bh / p.heads, h = bh - b * p.heads;
    const int nchunk = (p.seqlen + C - 1) / C;
    // chunk of loop step i: forwards, or backwards in the reverse pass
    auto chunk_of = [&](int i) { return MODE == 2 ? nchunk - 1 - i : i; };

    // The CTA's threads copy a chunk's rows and its block, one commit group per chunk.
    const int tid = threadIdx.x, hk = h / (p.heads / p.qk_heads);
    const size_t krow = size_t(p.qk_heads) * p.N, vrow = size_t(p.heads) * p.P;
    const size_t koff = size_t(b) * p.seqlen * krow + size_t(hk) * p.N;
    const size_t voff = size_t(b) * p.seqlen * vrow + size_t(h) * p.P + slice * NW * 16;
    auto copy_rows = [&](unsigned dst, int rowbytes, const auto *src, size_t stride, auto width, int limit, int t0) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
        constexpr int E = 16 / sizeof(T), CR = decltype(width)::value / E;      // values per copy, copies per row
#pragma unroll
        for (int i = 0; i < (C * CR + Cfg::NT - 1) / Cfg::NT; ++i) {
            const int x = tid + Cfg::NT * i, r = x / CR, n = (x % CR) * E;
            if (C * CR % Cfg::NT == 0 || x < C * CR) {
                const bool ok = t0 + r < p.seqlen && n < limit;
                cp_async_16z(dst + r * rowbytes + n * int(sizeof(T)), src + (ok ? size_t(t0 + r) * stride + n : 0), ok);
            }
        }
    };
    auto issue = [&](int i) {
        if (i < nchunk) {
            const int c = chunk_of(i), t0 = c * C;
            const unsigned base = smem_u32(smem + (i & 3) * Cfg::STAGE);
            const std::integral_constant<int, NP> kw;
            const std::integral_constant<int, NW * 16> vw;
#pragma unroll
            for (int m = 0; m < KP; ++m) {
                copy_rows(base + Cfg::OFF_K + m * Cfg::PIECE, Cfg::KROW,
                          static_cast<const __nv_bfloat16 *>(p.k) + m * p.piece + koff, krow, kw, p.N, t0);
                copy_rows(base + Cfg::OFF_Q + m * Cfg::PIECE, Cfg::KROW,
                          static_cast<const __nv_bfloat16 *>(p.q) + m * p.piece + koff, krow, kw, p.N, t0);
            }
            copy_rows(base + Cfg::OFF_V, Cfg::VROW, static_cast<const Tv *>(p.v) + voff, vrow, vw, p.P - slice * NW * 16, t0);
            if constexpr (MODE != 0)
                copy_rows(base + Cfg::OFF_V2, Cfg::V2ROW, static_cast<const typename Cfg::Tv2 *>(p.v2) + voff, vrow, vw,
                          p.P - slice * NW * 16, t0);
            const unsigned char *blk = p.prep + (size_t(bh) * nchunk + c) * Cfg::Block::BYTES;
            for (int x = tid; x < Cfg::Block::BYTES / 16; x += Cfg::NT)
                cp_async_16z(base + Cfg::OFF_TRI + 16 * x, blk + 16 * x, true);
        }
        cp_async_commit();
    };
    // The sums over the warps' rows of loop step i, left in shared memory at its end.
    auto flush_sums = [&](int i) {
        const int t = chunk_of(i) * C + (lane & 15), m = lane >> 4;
        if (m >= Cfg::NRED || t >= p.seqlen) return;
        const float *red = reinterpret_cast<const float *>(smem + Cfg::OFF_RED + (i & 1) * Cfg::REDBUF) + m * NW * C;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) x += red[w * C + (lane & 15)];
        (m ? p.sum1 : p.sum0)[(size_t(slice) * p.batch * p.heads + bh) * p.seqlen + t] = x;
    };
#pragma unroll
    for (int i = 0; i < 3; ++i) issue(i);

    const int g = lane >> 2, t4 = lane & 3;
    const int p0 = slice * NW * 16 + warp * 16;           // the warp's first row
    const int nrow = p.P - p0;                             // its rows (<= 0: none, may exceed 16)
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
    if (p.h0 != nullptr)
        state_io([&](float &x, float &y, size_t off) {
            const float2 f = *reinterpret_cast<const float2 *>(p.h0 + sbase + off);
            x = f.x; y = f.y;
        });
    unsigned char *tile = smem + Cfg::OFF_OUT + warp * C * kOutRow;
    const unsigned bn = b_rows_n(lane, Cfg::KROW), bk = b_rows_k(lane, Cfg::KROW);
    const unsigned tn = tri_rows_n(lane), tk = tri_rows_k(lane);
    const size_t ostride = vrow;
    const int nbound = (p.seqlen + kDeltaSave - 1) / kDeltaSave + 1;       // boundaries, the end among them
    auto bound_at = [&](int x) { return (size_t(bh) * nbound + x) * p.P * p.N; };
    auto keep_state = [&](float *ck, int x) {
        float *base = ck + bound_at(x);
        state_io([&](float &u, float &v, size_t off) { *reinterpret_cast<float2 *>(base + off) = make_float2(u, v); });
    };
    // reverse pass: the kept state of boundary x into the warp's rows of shared memory, and
    // its inner product with the gradient
    unsigned char *strow = smem + Cfg::OFF_ST + warp * 16 * Cfg::STROW;
    auto fetch_state = [&](int x) {
        const float *base = p.ck + bound_at(x);
        for (int y = lane; y < 16 * (NP / 4); y += 32) {
            const int r = y / (NP / 4), n = (y % (NP / 4)) * 4;
            const bool ok = r < nrow && n < p.N;
            cp_async_16z(smem_u32(strow + r * Cfg::STROW + n * 4), base + (ok ? size_t(p0 + r) * p.N + n : 0), ok);
        }
    };
    auto dot_state = [&](int x) {
        cp_async_wait<0>();
        __syncwarp();
        float z0 = 0.f, z1 = 0.f;
#pragma unroll
        for (int j = 0; j < NP / 8; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float2 f = *reinterpret_cast<const float2 *>(strow + (g + 8 * r) * Cfg::STROW + (8 * j + 2 * t4) * 4);
                z0 = fmaf(f.x, s[j][2 * r], z0);
                z1 = fmaf(f.y, s[j][2 * r + 1], z1);
            }
        z0 += z1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z0 += __shfl_xor_sync(0xffffffffu, z0, o);
        if (lane == 0)
            p.zsum[(size_t(slice * NW + warp) * p.batch * p.heads + bh) * nbound + x] = z0;
        __syncwarp();
    };
    // sums over the warp's 16 rows of f[row][token], for the producer to add up
    auto token_sums = [&](const float (&f)[2][4], int buf, int m) {
        float *red = reinterpret_cast<float *>(smem + Cfg::OFF_RED + buf * Cfg::REDBUF) + (m * NW + warp) * C;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float u = f[n][0] + f[n][2], w = f[n][1] + f[n][3];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                u += __shfl_xor_sync(0xffffffffu, u, o);
                w += __shfl_xor_sync(0xffffffffu, w, o);
            }
            if (g == 0) *reinterpret_cast<float2 *>(red + 8 * n + 2 * t4) = make_float2(u, w);
        }
    };
    if (nrow <= 0) {                                       // rows past headdim: only the barriers
        if constexpr (MODE != 0) {
            const float zero[2][4] = {};
#pragma unroll
            for (int m = 0; m < 2 * Cfg::NRED; ++m) token_sums(zero, m & 1, m >> 1);
        }
        if constexpr (MODE == 2)
            for (int x = lane; x < nbound; x += 32)
                p.zsum[(size_t(slice * NW + warp) * p.batch * p.heads + bh) * nbound + x] = 0.f;
        for (int i = 0; i < nchunk; ++i) {
            cp_async_wait<2>();
            __syncthreads();
            issue(i + 3);
        }
        cp_async_wait<0>();
        if constexpr (MODE != 0) __syncthreads();
        return;
    }
    if constexpr (MODE == 2) {
        fetch_state(nbound - 1);
        cp_async_commit();
    }

    for (int i = 0; i < nchunk; ++i) {
        const int c = chunk_of(i);
        cp_async_wait<2>();
        __syncthreads();
        const unsigned char *stage = smem + (i & 3) * Cfg::STAGE;
        const unsigned char *tri = stage + Cfg::OFF_TRI;
        const float *vec = reinterpret_cast<const float *>(tri + Cfg::Block::OFF_VEC);
        const unsigned kbase = smem_u32(stage + Cfg::OFF_K), qbase = smem_u32(stage + Cfg::OFF_Q), tbase = smem_u32(tri);
        const size_t tok0 = (size_t(b) * p.seqlen + size_t(c) * C) * p.heads + h;
        const int ntok = min(C, p.seqlen - c * C);
        constexpr int CS = kDeltaSave / C;
        float er[2][4];
        if constexpr (MODE == 1) if (c % CS == 0) keep_state(p.ck, c / CS);
        if constexpr (MODE == 2) {
            const float *ep = p.e + tok0 * p.P + p0;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int tok = 8 * n + 2 * t4 + (m & 1), row = g + 8 * (m >> 1);
                    er[n][m] = tok < ntok && row < nrow ? ep[size_t(tok) * ostride + row] : 0.f;
                }
            if (c % CS == CS - 1 || c == nchunk - 1) {
                keep_state(p.dck, c / CS + 1);
                dot_state(c / CS + 1);
            }
            if (c % CS == 0) fetch_state(c / CS);          // in the commit group of issue()
        }
        issue(i + 3);
        if constexpr (MODE != 0) if (i > 0 && warp == 0) flush_sums(i - 1);

        // S K^T, and S Q^T for y
        float sk[2][4], sks[2][4], sq[2][4], sqs[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) { zero4(sk[n]); zero4(sks[n]); zero4(sq[n]); zero4(sqs[n]); }
#pragma unroll
        for (int j = 0; j < NP / 16; ++j) {
            unsigned A[3][4], kb[KP][4];
            split_tiles<3>(s[2 * j], s[2 * j + 1], A);
#pragma unroll
            for (int m = 0; m < KP; ++m) ldsm4(kb[m], kbase + m * Cfg::PIECE + bn + j * 32);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma_pieces<3, KP>(sk[n], sks[n], A, kb, n);
            if constexpr (MODE != 2) {
                unsigned qb[KP][4];
#pragma unroll
                for (int m = 0; m < KP; ++m) ldsm4(qb[m], qbase + m * Cfg::PIECE + bn + j * 32);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    unsigned Ao[PO][4];
#pragma unroll
                    for (int m = 0; m < PO; ++m)
#pragma unroll
                        for (int r = 0; r < 4; ++r) Ao[m][r] = A[m][r];
                    mma_pieces<PO, KP>(sq[n], sqs[n], Ao, qb, n);
                }
            }
        }
        float v[2][4], x[2][4], du[2][4], gam[2][2], bet[2][2];
        load_tok_tile<Tv>(stage + Cfg::OFF_V + warp * 16 * int(sizeof(Tv)), Cfg::VROW, lane, v);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float2 f = *reinterpret_cast<const float2 *>(vec + (MODE == 2 ? 3 * C : 0) + 8 * n + 2 * t4);
            const float2 w = *reinterpret_cast<const float2 *>(vec + 2 * C + 8 * n + 2 * t4);
            gam[n][0] = f.x; gam[n][1] = f.y; bet[n][0] = w.x; bet[n][1] = w.y;
        }
        if constexpr (MODE != 2) {
            // R = v - gam S k;  e = R + (T - I) R
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) x[n][m] = fmaf(-gam[n][m & 1], sk[n][m] + sks[n][m], v[n][m]);
        } else {
            // rhs = end (dS k) + Pm^T dO, times beta;  w = rhs + (T - I)^T rhs
            float lo[2][4], los[2][4];
            unsigned A[Cfg::F32V ? 3 : 1][4], pb[3][4];
            split_tiles<Cfg::F32V ? 3 : 1>(v[0], v[1], A);
#pragma unroll
            for (int m = 0; m < 3; ++m) ldsm4_t(pb[m], tbase + (2 + m) * kTri + tk);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                zero4(lo[n]); zero4(los[n]);
                mma_pieces<Cfg::F32V ? 3 : 1, 3>(lo[n], los[n], A, pb, n);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    du[n][m] = fmaf(gam[n][m & 1], sk[n][m] + sks[n][m], lo[n][m] + los[n][m]);
                    x[n][m] = bet[n][m & 1] * du[n][m];
                }
            }
        }
        {
            unsigned A[2][4], tb[2][4];
            split_tiles<2>(x[0], x[1], A);
            float d[2][4], ds[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if constexpr (MODE == 2) ldsm4_t(tb[m], tbase + m * kTri + tk);
                else ldsm4(tb[m], tbase + m * kTri + tn);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                zero4(d[n]); zero4(ds[n]);
                mma_pieces<2, 2>(d[n], ds[n], A, tb, n);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) x[n][m] += d[n][m] + ds[n][m];
        }
        // the state's update: operand A1 against k (and in the reverse pass A2 against q)
        const float glast = vec[5 * C];
        unsigned A1[3][4];
        float w[2][4];
        if constexpr (MODE != 2) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 f = *reinterpret_cast<const float2 *>(vec + 4 * C + 8 * n + 2 * t4);
                w[n][0] = f.x * x[n][0]; w[n][1] = f.y * x[n][1]; w[n][2] = f.x * x[n][2]; w[n][3] = f.y * x[n][3];
            }
            split_tiles<3>(w[0], w[1], A1);
#pragma unroll
            for (int j = 0; j < NP / 16; ++j) {
                unsigned kb[KP][4];
#pragma unroll
                for (int m = 0; m < KP; ++m) ldsm4_t(kb[m], kbase + m * Cfg::PIECE + bk + j * 32);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float d[4], ds[4];
                    zero4(d); zero4(ds);
                    mma_pieces<3, KP>(d, ds, A1, kb, n);
#pragma unroll
                    for (int m = 0; m < 4; ++m) s[2 * j + n][m] = fmaf(glast, s[2 * j + n][m], d[m] + ds[m]);
                }
            }
        } else {
            unsigned A2[3][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 f = *reinterpret_cast<const float2 *>(vec + 8 * n + 2 * t4);
                w[n][0] = -f.x * x[n][0]; w[n][1] = -f.y * x[n][1]; w[n][2] = -f.x * x[n][2]; w[n][3] = -f.y * x[n][3];
            }
            split_tiles<3>(w[0], w[1], A1);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float2 f = *reinterpret_cast<const float2 *>(vec + C + 8 * n + 2 * t4);
                w[n][0] = f.x * v[n][0]; w[n][1] = f.y * v[n][1]; w[n][2] = f.x * v[n][2]; w[n][3] = f.y * v[n][3];
            }
            split_tiles<3>(w[0], w[1], A2);
#pragma unroll
            for (int j = 0; j < NP / 16; ++j) {
                unsigned kb[KP][4], qb[KP][4];
#pragma unroll
                for (int m = 0; m < KP; ++m) {
                    ldsm4_t(kb[m], kbase + m * Cfg::PIECE + bk + j * 32);
                    ldsm4_t(qb[m], qbase + m * Cfg::PIECE + bk + j * 32);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float d[4], ds[4];
                    zero4(d); zero4(ds);
                    mma_pieces<3, KP>(d, ds, A1, kb, n);
                    mma_pieces<3, KP>(d, ds, A2, qb, n);
#pragma unroll
                    for (int m = 0; m < 4; ++m) s[2 * j + n][m] = fmaf(glast, s[2 * j + n][m], d[m] + ds[m]);
                }
            }
        }
        if constexpr (MODE != 2) {
            // y = scale gam S q + Pm (beta e)
            unsigned A[PO][4], pb[PO][4];
            float o[2][4], os[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                w[n][0] = bet[n][0] * x[n][0]; w[n][1] = bet[n][1] * x[n][1];
                w[n][2] = bet[n][0] * x[n][2]; w[n][3] = bet[n][1] * x[n][3];
            }
            split_tiles<PO>(w[0], w[1], A);
#pragma unroll
            for (int m = 0; m < PO; ++m) ldsm4(pb[m], tbase + (2 + m) * kTri + tn);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                zero4(o[n]); zero4(os[n]);
                mma_pieces<PO, PO>(o[n], os[n], A, pb, n);
                const float2 f = *reinterpret_cast<const float2 *>(vec + C + 8 * n + 2 * t4);
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    o[n][m] = fmaf(m & 1 ? f.y : f.x, sq[n][m] + sqs[n][m], o[n][m] + os[n][m]);
            }
            if constexpr (MODE == 0) {
                store_tok_tile<Tout>(static_cast<Tout *>(p.y) + tok0 * p.P + p0, ostride, ntok, nrow, tile, lane, o);
            } else {
                store_tok_tile<float>(p.e + tok0 * p.P + p0, ostride, ntok, nrow, tile, lane, x);
                float dy[2][4];
                load_tok_tile<typename Cfg::Tv2>(stage + Cfg::OFF_V2 + warp * 16 * int(sizeof(typename Cfg::Tv2)),
                                                 Cfg::V2ROW, lane, dy);
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int m = 0; m < 4; ++m) dy[n][m] *= o[n][m];
                token_sums(dy, i & 1, 0);
            }
        } else {
            // du = rhs - (n / beta)^T w, the gradient of beta e: with e it gives beta's
            unsigned A[2][4], nb[2][4];
            float vv[2][4];
            split_tiles<2>(x[0], x[1], A);
#pragma unroll
            for (int m = 0; m < 2; ++m) ldsm4_t(nb[m], tbase + (2 + PO + m) * kTri + tk);
            load_tok_tile<typename Cfg::Tv2>(stage + Cfg::OFF_V2 + warp * 16 * int(sizeof(typename Cfg::Tv2)), Cfg::V2ROW,
                                             lane, vv);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float d[4], ds[4];
                zero4(d); zero4(ds);
                mma_pieces<2, 2>(d, ds, A, nb, n);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    du[n][m] = er[n][m] * (du[n][m] - (d[m] + ds[m]));
                    vv[n][m] *= x[n][m];
                }
            }
            token_sums(vv, i & 1, 0);
            token_sums(du, i & 1, 1);
            if (p.w != nullptr) store_tok_tile<float>(p.w + tok0 * p.P + p0, ostride, ntok, nrow, tile, lane, x);
            store_tok_tile<Tout>(static_cast<Tout *>(p.y) + tok0 * p.P + p0, ostride, ntok, nrow, tile, lane, x);
        }
    }
    cp_async_wait<0>();
    if constexpr (MODE != 0) {
        __syncthreads();
        if (warp == 0) flush_sums(nchunk - 1);
    }
    if constexpr (MODE == 1) keep_state(p.ck, nbound - 1);
    if constexpr (MODE == 2) dot_state(0);
    if (p.hN != nullptr)
        state_io([&](float &x, float &y, size_t off) {
            *reinterpret_cast<float2 *>(p.hN + sbase + off) = make_float2(x, y);
        });
}

}  // namespace ssm
