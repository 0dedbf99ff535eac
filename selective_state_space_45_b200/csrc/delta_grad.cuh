// delta_grad.cuh -- the gradients of q, k, a and beta of the gated delta rule, one chunk of
// 64 tokens and one key head per CTA, all chunks in parallel.
//
// The two passes of delta_rule.cuh leave, for every value head, e and w per token (w = the
// gradient of v) and the state S and its gradient dS at the chunk's two ends.  With S0 the
// state before the chunk, dE the gradient of the state behind it, u = beta e and
//     M1(t,s) = r(t,s) (dy_t.u_s)  for s <= t,     M2(t,s) = r(t,s) (w_t.u_s)  for s < t
// the chunk's gradients are
//     dq_t = scale (gam_t S0^T dy_t + sum_s M1(t,s) k_s)
//     dk_s = end_s dE^T u_s + scale sum_t M1(t,s) q_t - gam_s S0^T w_s - sum_t (M2 + M2^T)(s,t) k_t
// summed over the value heads that share the key head, in their order.  The gradient of a is
// <dS', S'>, S' the state after its decay; between tokens it changes by dy_t.y_t - v_t.w_t
// (q_t.dq_t - v_t.dv_t), so
//     da_t = <dS, S>(chunk's end) + sum_{t'>=t} (dy.y - v.w)_t'
//          = <dS, S>(chunk's start) - sum_{t'<t} (dy.y - v.w)_t'
// with the inner products taken afresh every 64 tokens: at most 32 terms are summed.
//
// Four warps with 16 tokens (rows) each, and with 64 columns of the state in shared memory four
// more that take the upper 32 of them: every product on the tensor cores with scaled fp16
// operands, here two pieces of each for fp32 gradients; delta_grad16.cuh is the form for bf16
// gradients (one piece: 2^-12 against their 2^-9).  Bound by the loads' latency and the
// conversions: 3 x 1021 tokens, 8 heads of 128 x 64 took 161 us with four warps and batches of
// two loads, about 130 so (one CTA per SM by shared memory either way).
// The token-by-token matrices never leave the registers: each is formed in the layout of an
// accumulator whose rows are the rows it is then used with (dy e^T for dq, e dy^T, e w^T and
// w e^T for dk), so that it becomes the next product's A operand as it stands, and tiles off
// the triangle are skipped; every warp has ten of them.  The largest magnitudes that set the
// scales come from the passes.
#pragma once

#include "delta_rule.cuh"

namespace ssm {

struct DeltaGradArgs {
    const void *dy;
    const float *a, *beta, *e, *w;     // e, w and the states as the passes leave them
    const unsigned char *rows, *prep;  // k and q as operands, and the chunk blocks (their scales)
    size_t block;                      // bytes of a chunk block
    const float *ck, *dck;             // states and their gradients at the boundaries
    const unsigned char *e16, *w16, *y16, *s16, *d16;      // bf16 gradients: the same as fp16 tiles
    unsigned *timeouts;
    const float *dyy, *edu, *vw;       // [zparts][batch][heads][seqlen]
    const float *zsum;                 // [zparts][batch][heads][boundaries]
    const unsigned *smax, *dsmax;      // [batch][heads][boundaries][zparts]
    const unsigned *emax, *wmax, *ymax;// [batch][heads][chunks of 32][zparts]
    float *part;                       // heads that share a key head: running sums of dq, dk, [2][tokens][qk_heads][N]
    void *dq, *dk;
    float *da, *dbeta;
    int batch, seqlen, heads, qk_heads, P, N, zparts;
    float scale;
};

constexpr int kGradC = 64, kGradN = 64;        // tokens per CTA, state columns per pass

// PW: headdim padded to 64 or 128; NP: dstate padded; KP: pieces of k and q; PG: of the others.
template <int NP_, int PW_, int KP_> struct GradCfg {
    static constexpr int NP = NP_, PW = PW_, KP = KP_, PG = 2;
    static constexpr int W = NP < kGradN ? NP : kGradN, NT = 128 * (W / 32);
    static constexpr int PROW = PW * 2 + 16, NROW = W * 2 + 16, TROW = kGradC * 2 + 16;      // padded rows (bytes)
    static constexpr int TOK = kGradC * PROW, TT = PW * TROW, ST = PW * NROW, KT = kGradC * NROW;
    static constexpr int OFF_Y = 0, OFF_E = OFF_Y + PG * TOK, OFF_W = OFF_E + PG * TT;
    static constexpr int OFF_S = OFF_W + PG * TT, OFF_D = OFF_S + PG * ST;
    static constexpr int OFF_K = OFF_D + PG * ST, OFF_Q = OFF_K + KP * KT;
    static constexpr int OFF_VEC = OFF_Q + KP * KT;
    static constexpr int SMEM_BYTES = OFF_VEC + 6 * kGradC * 4 + 16;
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT) delta_grad_kernel(const DeltaGradArgs p) {
    constexpr int C = kGradC, NP = Cfg::NP, PW = Cfg::PW, KP = Cfg::KP, PG = Cfg::PG, W = Cfg::W, NT = Cfg::NT;
    using Rows = DeltaRows<NP, KP>;
    extern __shared__ __align__(128) unsigned char delta_smem[];
    unsigned char *smem = delta_smem;
    float *Gh = reinterpret_cast<float *>(smem + Cfg::OFF_VEC), *Gl = Gh + C, *gam = Gl + C, *bet = gam + C;
    float *bend = bet + C, *dtok = bend + C;
    double *half = reinterpret_cast<double *>(dtok + C);
    const int tid = threadIdx.x, lane = tid & 31, rt = (tid >> 5) & 3, j0 = tid >> 7, g = lane >> 2, t4 = lane & 3;
    const int nchunk = (p.seqlen + C - 1) / C, nbound = nchunk + 1, nck = (p.seqlen + kDeltaC - 1) / kDeltaC;
    const int c = int(blockIdx.x % unsigned(nchunk)), bk = int(blockIdx.x / unsigned(nchunk));
    const int b = bk / p.qk_heads, hk = bk - b * p.qk_heads;
    const int t0 = c * C, nt = min(C, p.seqlen - t0), group = p.heads / p.qk_heads;
    const int c32 = 2 * c, n32 = min(2, nck - c32);
    const size_t all = size_t(p.batch) * p.heads, krow = size_t(p.qk_heads) * p.N, vrow = size_t(p.heads) * p.P;
    const size_t k0 = (size_t(b) * p.seqlen + t0) * krow + size_t(hk) * p.N;

    // 1 / scales of k and q in the chunk's halves
    float ick[2], icq[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int cc = c32 + (x < n32 ? x : 0);
        const float *one = reinterpret_cast<const float *>(p.prep + ((size_t(b) * p.heads + hk * group) * nck + cc) * p.block +
                                                           DeltaBlock::OFF_VEC) + kVecScalars * kDeltaC;
        ick[x] = 1.f / one[kCk];         // powers of two: exact
        icq[x] = 1.f / one[kCq];
    }
    const unsigned an = unsigned((16 * rt + (lane & 15)) * Cfg::PROW + (lane >> 4) * 16);      // A: this warp's rows
    const unsigned bp = b_rows_n(lane, Cfg::PROW), bn = b_rows_k(lane, Cfg::NROW);
    const unsigned at_ = b_rows_n(lane, Cfg::TROW) + 32 * rt, bt = b_rows_k(lane, Cfg::TROW);     // e, w: [headdim][token]

    for (int hg = 0; hg < group; ++hg) {
        const int h = hk * group + hg;
        const size_t bh = size_t(b) * p.heads + h;
        const size_t v0 = (size_t(b) * p.seqlen + t0) * vrow + size_t(h) * p.P;
        // scales: the largest magnitudes over the rows' warps (and the chunk's halves); at most
        // 8 and 16 values each
        auto max_at = [&](const unsigned *m, size_t first, int n) { return lane < n ? __ldg(m + first + lane) : 0u; };
        unsigned big[5] = {max_at(p.smax, (bh * nbound + c) * p.zparts, p.zparts),
                           max_at(p.dsmax, (bh * nbound + c + 1) * p.zparts, p.zparts),
                           max_at(p.emax, (bh * nck + c32) * p.zparts, n32 * p.zparts),
                           max_at(p.wmax, (bh * nck + c32) * p.zparts, n32 * p.zparts),
                           max_at(p.ymax, (bh * nck + c32) * p.zparts, n32 * p.zparts)};
        // threads 0..63: their token's gates and sums
        const size_t gate = (size_t(b) * p.seqlen + t0 + (tid & 63)) * p.heads + h;
        float av = 0.f, bv = 0.f, dyy = 0.f, db = 0.f, z = 0.f;
        const bool front = 2 * tid < nt;
        if (tid < nt) {
            av = fmaxf(p.a[gate], -1e4f);
            bv = p.beta[gate];
#pragma unroll 4
            for (int s = 0; s < p.zparts; ++s) {
                const size_t x = (s * all + bh) * p.seqlen + t0 + tid;
                dyy += p.dyy[x] - p.vw[x];
                db += p.edu[x];
            }
#pragma unroll 4
            for (int s = 0; s < p.zparts; ++s) z += p.zsum[(s * all + bh) * nbound + c + (front ? 0 : 1)];
        }
#pragma unroll
        for (int x = 0; x < 5; ++x) big[x] = __reduce_max_sync(0xffffffffu, big[x]);
        const Pow2 cS = pow2_for(big[0]), cD = pow2_for(big[1]), cE = pow2_for(big[2]), cW = pow2_for(big[3]), cY = pow2_for(big[4]);
        __syncthreads();                 // the last head's tiles and vectors are done with

        // dy as an operand [token][headdim], e and w as [headdim][token]
        const float *dyp = static_cast<const float *>(p.dy) + v0;
        constexpr int CP = PW / 8;
#pragma unroll 4
        for (int i = tid; i < C * CP; i += NT) {
            const int r = i / CP, x = (i % CP) * 8;
            float f[8] = {};
            if (r < nt && x < p.P) load8(dyp + size_t(r) * vrow + x, f);
            unsigned u[4][PG];
#pragma unroll
            for (int y = 0; y < 4; ++y) split_f16<PG>(f2(f[2 * y], f[2 * y + 1]), cY.c, u[y]);
#pragma unroll
            for (int y = 0; y < PG; ++y)
                *reinterpret_cast<uint4 *>(smem + Cfg::OFF_Y + y * Cfg::TOK + r * Cfg::PROW + x * 2) =
                    make_uint4(u[0][y], u[1][y], u[2][y], u[3][y]);
        }
        // what a lane of the passes held, two rows of two neighbouring columns, into a tile of rows
        auto put = [&](unsigned char *to, int piece, int rowbytes, float4 f, float scale) {
            unsigned x[PG], y[PG];
            split_f16<PG>(f2(f.x, f.y), scale, x);
            split_f16<PG>(f2(f.z, f.w), scale, y);
#pragma unroll
            for (int i = 0; i < PG; ++i) {
                *reinterpret_cast<unsigned *>(to + i * piece + g * rowbytes + 4 * t4) = x[i];
                *reinterpret_cast<unsigned *>(to + i * piece + (g + 8) * rowbytes + 4 * t4) = y[i];
            }
        };
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = tid >> 5; i < 2 * (PW / 16) * 4; i += NT / 32) {      // (half, 16 rows, 8 tokens)
            const int n = i & 3, rb = (i >> 2) % (PW / 16), hf = i / (PW / 4);
            const bool ok = hf < n32 && 16 * rb < p.P;
            const size_t from = ((((bh * nck + c32 + hf) * p.zparts + rb) * 4 + n) * 32 + lane) * 4;
            const float4 fe = ok ? __ldg(reinterpret_cast<const float4 *>(p.e + from)) : none;
            const float4 fw = ok ? __ldg(reinterpret_cast<const float4 *>(p.w + from)) : none;
            unsigned char *to = smem + 16 * rb * Cfg::TROW + 64 * hf + 16 * n;
            put(to + Cfg::OFF_E, Cfg::TT, Cfg::TROW, fe, cE.c);
            put(to + Cfg::OFF_W, Cfg::TT, Cfg::TROW, fw, cW.c);
        }
        // decays: prefix sums of a in 64 bits, kept as pairs of floats (a below -1e4 counts as
        // -1e4: its exponential is 0 either way, and the sums stay finite)
        double G = av;
        if (tid < C) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, G, o);
                if (lane >= o) G += u;
            }
            if (lane == 31) half[tid >> 5] = G;
        }
        __syncthreads();
        if (tid < C) {
            const double Gend = half[0] + half[1];
            if (tid >= 32) G += half[0];
            Gh[tid] = float(G);
            Gl[tid] = float(G - double(float(G)));
            gam[tid] = expf(float(G));
            bet[tid] = bv;
            bend[tid] = bv * expf(float(Gend - G));
            dtok[tid] = dyy;
        }
        // The token-by-token matrices of this warp's rows, in four tiles of 16 columns.
        const unsigned sy = smem_u32(smem + Cfg::OFF_Y), se = smem_u32(smem + Cfg::OFF_E), sw = smem_u32(smem + Cfg::OFF_W);
        float x1[4][2][4], x2[4][2][4], x3[4][2][4], x4[2][4];   // dy e^T; e dy^T; w e^T, e w^T past the diagonal; e w^T on it
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < 2; ++n) { zero4(x1[u][n]); zero4(x2[u][n]); zero4(x3[u][n]); }
        zero4(x4[0]); zero4(x4[1]);
#pragma unroll
        for (int k = 0; k < PW / 16; ++k) {
            unsigned ay[PG][4], ae[PG][4], aw[PG][4];
#pragma unroll
            for (int i = 0; i < PG; ++i) {
                ldsm4(ay[i], sy + i * Cfg::TOK + an + k * 32);
                ldsm4_t(ae[i], se + i * Cfg::TT + at_ + 16 * k * Cfg::TROW);
                ldsm4_t(aw[i], sw + i * Cfg::TT + at_ + 16 * k * Cfg::TROW);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                unsigned be[PG][4], by[PG][4], bw[PG][4];
                const unsigned at = 16 * u * Cfg::PROW + bp + k * 32, tt = 16 * k * Cfg::TROW + bt + 32 * u;
                if (u <= rt) {
#pragma unroll
                    for (int i = 0; i < PG; ++i) ldsm4_t(be[i], se + i * Cfg::TT + tt);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma_pieces<PG, PG>(x1[u][n], ay, be, n);
                        mma_pieces<PG, PG>(x3[u][n], aw, be, n);
                    }
                }
                if (u >= rt) {
#pragma unroll
                    for (int i = 0; i < PG; ++i) {
                        ldsm4(by[i], sy + i * Cfg::TOK + at);
                        ldsm4_t(bw[i], sw + i * Cfg::TT + tt);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma_pieces<PG, PG>(x2[u][n], ae, by, n);
                        if (u == rt) mma_pieces<PG, PG>(x4[n], ae, bw, n);
                        else mma_pieces<PG, PG>(x3[u][n], ae, bw, n);
                    }
                }
            }
        }
        __syncthreads();
        // times the decays, beta and the scales taken back out: M1 / ck for dq; M1^T scale / cq
        // and -(M2 + M2^T) / ck for dk
        float m1 = 0.f, m2 = 0.f;
        const float fye = cY.inv * cE.inv, fwe = cW.inv * cE.inv;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int r = 16 * rt + g + 8 * (m >> 1), q = 16 * u + 8 * n + 2 * t4 + (m & 1);
                    const float gd = (Gh[r] - Gh[q]) + (Gl[r] - Gl[q]);
                    const float up = ex2_approx((q <= r ? gd : -gd) * kLog2e);     // r(the later, the earlier)
                    const float b0 = bet[q < r ? q : r], back = u < 2 ? ick[0] : ick[1], backq = u < 2 ? icq[0] : icq[1];
                    const float d = up * b0;
                    x1[u][n][m] = q <= r ? x1[u][n][m] * (d * p.scale * fye * back) : 0.f;
                    x2[u][n][m] = q >= r ? x2[u][n][m] * (d * p.scale * fye * backq) : 0.f;
                    const float w3 = (u == rt && q > r) ? x4[n][m] : x3[u][n][m];
                    x3[u][n][m] = q != r ? -w3 * (d * fwe * back) : 0.f;
                    m1 = fmaxf(m1, fabsf(x1[u][n][m]));
                    m2 = fmaxf(m2, fmaxf(fabsf(x2[u][n][m]), fabsf(x3[u][n][m])));
                }
        const Pow2 c1 = pow2_for(warp_max_bits(m1)), c2 = pow2_for(warp_max_bits(m2));
        unsigned a1[4][PG][4], a2[4][PG][4], a3[4][PG][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            split_tiles<PG>(x1[u][0], x1[u][1], c1.c, a1[u]);
            split_tiles<PG>(x2[u][0], x2[u][1], c2.c, a2[u]);
            split_tiles<PG>(x3[u][0], x3[u][1], c2.c, a3[u]);
        }
        float fq[2], fw[2], fe[2];       // row factors of the products with the states
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = 16 * rt + g + 8 * r;
            fq[r] = p.scale * gam[t] * (cY.inv * cS.inv);
            fw[r] = -gam[t] * (cW.inv * cS.inv);
            fe[r] = bend[t] * (cE.inv * cD.inv);
        }

        const float *S0 = p.ck + (bh * nbound + c) * p.zparts * (NP * 16);
        const float *dE = p.dck + (bh * nbound + c + 1) * p.zparts * (NP * 16);
        for (int n0 = 0; n0 < NP; n0 += W) {
            if (n0 > 0) __syncthreads();
            // this pass's columns of the states and of k and q
            constexpr int CN = W / 8;
#pragma unroll 4
            for (int i = tid >> 5; i < (PW / 16) * CN; i += NT / 32) {     // (16 rows, 8 columns)
                const int j = i % CN, rb = i / CN;
                const bool ok = 16 * rb < p.P && n0 + 8 * j < NP;
                const size_t from = ((size_t(rb) * (NP / 8) + n0 / 8 + j) * 32 + lane) * 4;
                const float4 fs = ok ? __ldg(reinterpret_cast<const float4 *>(S0 + from)) : none;
                const float4 fd = ok ? __ldg(reinterpret_cast<const float4 *>(dE + from)) : none;
                unsigned char *to = smem + 16 * rb * Cfg::NROW + 16 * j;
                put(to + Cfg::OFF_S, Cfg::ST, Cfg::NROW, fs, cS.c);
                put(to + Cfg::OFF_D, Cfg::ST, Cfg::NROW, fd, cD.c);
            }
#pragma unroll 4
            for (int i = tid; i < C * CN; i += NT) {
                const int r = i / CN, x = (i % CN) * 8, half = r / kDeltaC;
                const unsigned char *src = p.rows + ((size_t(b) * p.qk_heads + hk) * nck + c32 + (half < n32 ? half : 0)) * Rows::BYTES +
                                           (r % kDeltaC) * Rows::ROW + (n0 + x) * 2;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int y = 0; y < KP; ++y) {
                        const uint4 w = half < n32 && n0 + x < NP
                                            ? __ldg(reinterpret_cast<const uint4 *>(src + (m * KP + y) * Rows::PIECE))
                                            : make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(smem + (m ? Cfg::OFF_Q : Cfg::OFF_K) + y * Cfg::KT + r * Cfg::NROW + x * 2) = w;
                    }
            }
            __syncthreads();
            const unsigned sS = smem_u32(smem + Cfg::OFF_S), sD = smem_u32(smem + Cfg::OFF_D);
            const unsigned sk = smem_u32(smem + Cfg::OFF_K), sq = smem_u32(smem + Cfg::OFF_Q);
            // 32 columns per group of four warps
            float aq[4][4], ak[4][4], aw[4][4], ae[4][4], am[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) { zero4(aq[n]); zero4(ak[n]); zero4(aw[n]); zero4(ae[n]); zero4(am[n]); }
#pragma unroll
            for (int k = 0; k < PW / 16; ++k) {
                unsigned ay[PG][4], aE[PG][4], aW[PG][4];
#pragma unroll
                for (int i = 0; i < PG; ++i) {
                    ldsm4(ay[i], sy + i * Cfg::TOK + an + k * 32);
                    ldsm4_t(aE[i], se + i * Cfg::TT + at_ + 16 * k * Cfg::TROW);
                    ldsm4_t(aW[i], sw + i * Cfg::TT + at_ + 16 * k * Cfg::TROW);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    unsigned bS[PG][4], bD[PG][4];
                    const unsigned at = 16 * k * Cfg::NROW + bn + j0 * 64 + j * 32;
#pragma unroll
                    for (int i = 0; i < PG; ++i) {
                        ldsm4_t(bS[i], sS + i * Cfg::ST + at);
                        ldsm4_t(bD[i], sD + i * Cfg::ST + at);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma_pieces<PG, PG>(aq[2 * j + n], ay, bS, n);
                        mma_pieces<PG, PG>(aw[2 * j + n], aW, bS, n);
                        mma_pieces<PG, PG>(ae[2 * j + n], aE, bD, n);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    unsigned bK[KP][4], bQ[KP][4];
                    const unsigned at = 16 * u * Cfg::NROW + bn + j0 * 64 + j * 32;
#pragma unroll
                    for (int i = 0; i < KP; ++i) ldsm4_t(bK[i], sk + i * Cfg::KT + at);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if (u <= rt) mma_pieces<PG, KP>(ak[2 * j + n], a1[u], bK, n);
                        mma_pieces<PG, KP>(am[2 * j + n], a3[u], bK, n);
                    }
                    if (u >= rt) {
#pragma unroll
                        for (int i = 0; i < KP; ++i) ldsm4_t(bQ[i], sq + i * Cfg::KT + at);
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_pieces<PG, KP>(am[2 * j + n], a2[u], bQ, n);
                    }
                }
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int t = 16 * rt + g + 8 * r, col = n0 + 32 * j0 + 8 * n + 2 * t4;
                    if (t >= nt || col >= p.N) continue;
                    const size_t off = k0 + size_t(t) * krow + col;
                    float2 q, k;
                    q.x = fmaf(c1.inv, ak[n][2 * r], fq[r] * aq[n][2 * r]);
                    q.y = fmaf(c1.inv, ak[n][2 * r + 1], fq[r] * aq[n][2 * r + 1]);
                    k.x = fmaf(c2.inv, am[n][2 * r], fmaf(fw[r], aw[n][2 * r], fe[r] * ae[n][2 * r]));
                    k.y = fmaf(c2.inv, am[n][2 * r + 1], fmaf(fw[r], aw[n][2 * r + 1], fe[r] * ae[n][2 * r + 1]));
                    float2 *pq = reinterpret_cast<float2 *>(p.part + off);
                    float2 *pk = reinterpret_cast<float2 *>(p.part + size_t(p.batch) * p.seqlen * krow + off);
                    if (hg > 0) { q = fadd2(*pq, q); k = fadd2(*pk, k); }
                    if (hg + 1 < group) {
                        *pq = q;
                        *pk = k;
                    } else {
                        *reinterpret_cast<float2 *>(static_cast<float *>(p.dq) + off) = q;
                        *reinterpret_cast<float2 *>(static_cast<float *>(p.dk) + off) = k;
                    }
                }
        }
        if (tid < nt) {
            if (front) for (int x = 0; x < tid; ++x) z -= dtok[x];
            else for (int x = nt - 1; x >= tid; --x) z += dtok[x];
            p.da[gate] = z;
            p.dbeta[gate] = db;
        }
    }
}

}  // namespace ssm
