// delta_grad16.cuh -- the gradients of q, k, a and beta of the gated delta rule behind bf16
// gradients: the sums of delta_grad.cuh, with operands that the passes have already left as
// scaled fp16 tiles of this kernel's shared memory.
//
// A CTA (a chunk of 64 tokens of one key head) starts ten bulk copies per value head and waits
// once: nothing is loaded, converted or stored by its threads on the way.  Converting fp32
// operands here instead took 4000 of 6100 instructions a warp, and 446 us where this takes 296
// (8 x 2048 tokens, 24 heads over 24 key heads, headdim 64, dstate 128).  What is left is the
// latency of the copies and of dependent products, at two CTAs an SM.  A tile's scale is that of
// its part, 16 rows of headdim, which are one step of a product's inner index: before a step its
// A operand is multiplied with the power of two (at most 1) that brings the step's product to
// the smallest of the parts' scales.
#pragma once

#include "delta_grad.cuh"

namespace ssm {

// KP: fp16 pieces of k and q.  PW: headdim padded to 64 or 128.
template <int NP_, int PW_, int KP_> struct Grad16Cfg {
    static constexpr int NP = NP_, PW = PW_, KP = KP_, PARTS = PW / 16;
    using Rows = DeltaRows<NP, KP>;
    using S16 = State16<NP>;
    static constexpr int TOK = 2 * PARTS * kTok16;                            // [half][part] tiles
    static constexpr int OFF_E = 0, OFF_W = TOK, OFF_Y = 2 * TOK;
    static constexpr int OFF_S = 3 * TOK, OFF_D = OFF_S + PARTS * S16::BYTES;
    static constexpr int OFF_KQ = OFF_D + PARTS * S16::BYTES;                 // [half] k and q
    static constexpr int OFF_VEC = OFF_KQ + 2 * Rows::BYTES;
    static constexpr int OFF_OUT = OFF_VEC + 6 * kGradC * 4 + 32;             // per-warp output tiles
    static constexpr int SMEM_BYTES = OFF_OUT + 4 * kTok16;
    static constexpr int CTAS = SMEM_BYTES <= 113 * 1024 ? 2 : 1;
};

// 2^e as a float and, for e <= 0, as a pair of halves (0 below the smallest).
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(unsigned(min(max(e, -126), 127) + 127) << 23); }
__device__ __forceinline__ unsigned half2_exp2(int e) {
    const __half2 h = __float2half2_rn(exp2_int(e));
    return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ void mul_f16x2(unsigned (&o)[4], const unsigned (&a)[4], unsigned f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&a[i]), *reinterpret_cast<const __half2 *>(&f));
        o[i] = *reinterpret_cast<const unsigned *>(&h);
    }
}

template <class Cfg>
__global__ void __launch_bounds__(128, Cfg::CTAS) delta_grad16_kernel(const DeltaGradArgs p) {
    using Rows = typename Cfg::Rows;
    using S16 = typename Cfg::S16;
    constexpr int C = kGradC, NP = Cfg::NP, KP = Cfg::KP;
    extern __shared__ __align__(128) unsigned char delta_smem[];
    unsigned char *smem = delta_smem;
    float *Gh = reinterpret_cast<float *>(smem + Cfg::OFF_VEC), *Gl = Gh + C, *gam = Gl + C, *bet = gam + C;
    float *bend = bet + C, *dtok = bend + C;
    double *half = reinterpret_cast<double *>(dtok + C);
    uint64_t *bar = reinterpret_cast<uint64_t *>(half + 2);
    const int tid = threadIdx.x, lane = tid & 31, rt = tid >> 5, ht = rt >> 1, g = lane >> 2, t4 = lane & 3;
    const int nchunk = (p.seqlen + C - 1) / C, nbound = nchunk + 1, nck = (p.seqlen + kDeltaC - 1) / kDeltaC;
    const int c = int(blockIdx.x % unsigned(nchunk)), bk = int(blockIdx.x / unsigned(nchunk));
    const int b = bk / p.qk_heads, hk = bk - b * p.qk_heads;
    const int t0 = c * C, nt = min(C, p.seqlen - t0), group = p.heads / p.qk_heads;
    const int c32 = 2 * c, n32 = min(2, nck - c32), kp = (p.P + 15) / 16;
    const size_t all = size_t(p.batch) * p.heads, krow = size_t(p.qk_heads) * p.N;
    const size_t k0 = (size_t(b) * p.seqlen + t0) * krow + size_t(hk) * p.N;
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_fence_init();
    }
    auto zero = [&](int off, int bytes) {
        for (int x = tid; x < bytes / 16; x += 128) *reinterpret_cast<uint4 *>(smem + off + 16 * x) = make_uint4(0, 0, 0, 0);
    };
    // a chunk whose second half is past the end: that half is zeros
    if (n32 == 1) {
        zero(Cfg::OFF_E + Cfg::TOK / 2, Cfg::TOK / 2);
        zero(Cfg::OFF_W + Cfg::TOK / 2, Cfg::TOK / 2);
        zero(Cfg::OFF_Y + Cfg::TOK / 2, Cfg::TOK / 2);
        zero(Cfg::OFF_KQ + Rows::BYTES, Rows::BYTES);
    }
    if (kp < Cfg::PARTS) {               // parts past headdim: zeros
        const int n = Cfg::PARTS - kp;
        for (int hf = 0; hf < 2; ++hf) {
            zero(Cfg::OFF_E + hf * (Cfg::TOK / 2) + kp * kTok16, n * kTok16);
            zero(Cfg::OFF_W + hf * (Cfg::TOK / 2) + kp * kTok16, n * kTok16);
            zero(Cfg::OFF_Y + hf * (Cfg::TOK / 2) + kp * kTok16, n * kTok16);
        }
        zero(Cfg::OFF_S + kp * S16::BYTES, n * S16::BYTES);
        zero(Cfg::OFF_D + kp * S16::BYTES, n * S16::BYTES);
    }
    __syncthreads();
    auto copies = [&](int hg) {          // by one thread
        const size_t bh = size_t(b) * p.heads + hk * group + hg;
        const uint32_t tok = kp * kTok16, st = kp * S16::BYTES;
        mbar_arrive_expect_tx(bar, n32 * (3 * tok + (hg == 0 ? Rows::BYTES : 0)) + 2 * st);
        for (int hf = 0; hf < n32; ++hf) {
            const size_t at = (bh * nck + c32 + hf) * p.zparts * kTok16;
            unsigned char *to = smem + hf * (Cfg::TOK / 2);
            bulk_load(to + Cfg::OFF_E, p.e16 + at, tok, bar);
            bulk_load(to + Cfg::OFF_W, p.w16 + at, tok, bar);
            bulk_load(to + Cfg::OFF_Y, p.y16 + at, tok, bar);
            if (hg == 0)
                bulk_load(smem + Cfg::OFF_KQ + hf * Rows::BYTES,
                          p.rows + ((size_t(b) * p.qk_heads + hk) * nck + c32 + hf) * Rows::BYTES, Rows::BYTES, bar);
        }
        bulk_load(smem + Cfg::OFF_S, p.s16 + (bh * nbound + c) * p.zparts * S16::BYTES, st, bar);
        bulk_load(smem + Cfg::OFF_D, p.d16 + (bh * nbound + c + 1) * p.zparts * S16::BYTES, st, bar);
    };
    if (tid == 0) copies(0);

    // ldmatrix offsets.  e, w, dy tiles are [headdim][token], states [headdim][dstate]: both take
    // the transposing load.  A: this warp's 16 tokens; B: 16 tokens of a half, or 16 columns.
    const int ra = (lane >> 4) * 8 + (lane & 7), rb = (lane >> 3 & 1) * 8 + (lane & 7);
    const unsigned a_tok = ht * (Cfg::TOK / 2) + tok16_at(ra, (rt & 1) * 2 + (lane >> 3 & 1));
    const unsigned b_tok[2] = {unsigned(tok16_at(rb, lane >> 4)), unsigned(tok16_at(rb, 2 + (lane >> 4)))};
    const unsigned b_st = rb * S16::ROW, x_st = ((lane >> 4) * 16) ^ S16::flip(rb);
    const unsigned b_kq = b_rows_k(lane, Rows::ROW);
    const unsigned sbase = smem_u32(smem);

    bool alive = true;
    float ick[2], icq[2];                // 1 / scales of k and q in the chunk's halves
    for (int hg = 0; hg < group; ++hg) {
        const int h = hk * group + hg;
        const size_t bh = size_t(b) * p.heads + h;
        // Everything small at once: scales, and for threads 0..63 their token's gates and sums.
        if (hg == 0)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int cc = c32 + (x < n32 ? x : 0);
                const float *one = reinterpret_cast<const float *>(p.prep + ((size_t(b) * p.heads + h) * nck + cc) * p.block +
                                                                   DeltaBlock::OFF_VEC) + kVecScalars * kDeltaC;
                ick[x] = __ldg(one + kCk);
                icq[x] = __ldg(one + kCq);
            }
        unsigned bits[8];                                 // lane k: part k's largest magnitudes
        auto max_at = [&](const unsigned *m, size_t first) { return lane < kp ? __ldg(m + first + lane) : 0u; };
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const size_t at = (bh * nck + c32 + (x < n32 ? x : 0)) * p.zparts;
            bits[x] = max_at(p.ymax, at);
            bits[2 + x] = max_at(p.emax, at);
            bits[4 + x] = max_at(p.wmax, at);
        }
        bits[6] = max_at(p.smax, (bh * nbound + c) * p.zparts);
        bits[7] = max_at(p.dsmax, (bh * nbound + c + 1) * p.zparts);
        const size_t gate = (size_t(b) * p.seqlen + t0 + (tid & 63)) * p.heads + h;
        float av = 0.f, bv = 0.f, dyy = 0.f, db = 0.f, z = 0.f;
        const bool front = 2 * tid < nt;
        if (tid < nt) {
            av = __ldg(p.a + gate);
            bv = __ldg(p.beta + gate);
            float v[4][4];
            for (int s0 = 0; s0 < p.zparts; s0 += 4) {    // zparts is a multiple of 4
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const size_t x = ((s0 + s) * all + bh) * p.seqlen + t0 + tid;
                    v[s][0] = __ldg(p.dyy + x);
                    v[s][1] = __ldg(p.vw + x);
                    v[s][2] = __ldg(p.edu + x);
                    v[s][3] = __ldg(p.zsum + ((s0 + s) * all + bh) * nbound + c + (front ? 0 : 1));
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) { dyy += v[s][0] - v[s][1]; db += v[s][2]; z += v[s][3]; }
            }
            av = fmaxf(av, -1e4f);
        }
        if (hg == 0)
#pragma unroll
            for (int x = 0; x < 2; ++x) { ick[x] = 1.f / ick[x]; icq[x] = 1.f / icq[x]; }       // powers of two: exact
        // Scales as powers of two: per product the smallest over the parts (the products come out
        // times 2^it) and each part's distance to it.
        int ly[2], le[2], lw[2];
        auto log_scale = [&](unsigned m) { return int(__float_as_uint(pow2_for(m).c) >> 23) - 127; };
#pragma unroll
        for (int x = 0; x < 2; ++x) { ly[x] = log_scale(bits[x]); le[x] = log_scale(bits[2 + x]); lw[x] = log_scale(bits[4 + x]); }
        const int ls = log_scale(bits[6]), ld = log_scale(bits[7]);
        auto common = [&](int l, float &inv) {
            const int least = __reduce_min_sync(0xffffffffu, lane < kp ? l : 1 << 20);
            inv = exp2_int(-(least >> 1)) * exp2_int((least >> 1) - least);       // 0 when too small for a float
            return lane < kp ? half2_exp2(least - l) : 0u;
        };
        float i1[2], i2[2], i3[2], i4[2], i5, i6, i7;
        unsigned f1[2], f2x[2], f3[2], f4[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            f1[x] = common(ly[ht] + le[x], i1[x]);        // dy e^T
            f2x[x] = common(le[ht] + ly[x], i2[x]);       // e dy^T
            f3[x] = common(lw[ht] + le[x], i3[x]);        // w e^T
            f4[x] = common(le[ht] + lw[x], i4[x]);        // e w^T
        }
        const unsigned f5 = common(ly[ht] + ls, i5), f6 = common(lw[ht] + ls, i6), f7 = common(le[ht] + ld, i7);
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
        __syncthreads();
        if (!mbar_test(bar, hg & 1) && !mbar_wait(bar, hg & 1, kDeltaWaitCycles)) {
            alive = false;
            atomicAdd(p.timeouts, 1u);
        }

        // The token-by-token matrices of this warp's rows, in four tiles of 16 columns: dy e^T;
        // e dy^T; w e^T up to the diagonal and e w^T past it; e w^T on it.
        float x1[4][2][4], x2[4][2][4], x3[4][2][4], x4[2][4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < 2; ++n) { zero4(x1[u][n]); zero4(x2[u][n]); zero4(x3[u][n]); }
        zero4(x4[0]); zero4(x4[1]);
#pragma unroll 4
        for (int k = 0; k < Cfg::PARTS; ++k) {
            unsigned ay[1][4], ae[1][4], aw[1][4];
            const unsigned kt = sbase + k * kTok16;
            ldsm4_t(ay[0], kt + Cfg::OFF_Y + a_tok);
            ldsm4_t(ae[0], kt + Cfg::OFF_E + a_tok);
            ldsm4_t(aw[0], kt + Cfg::OFF_W + a_tok);
#pragma unroll
            for (int hu = 0; hu < 2; ++hu) {
                unsigned sy[1][4], se[1][4], sw[1][4], ew[1][4];
                if (hu <= ht) {
                    mul_f16x2(sy[0], ay[0], __shfl_sync(0xffffffffu, f1[hu], k));
                    mul_f16x2(sw[0], aw[0], __shfl_sync(0xffffffffu, f3[hu], k));
                }
                if (hu >= ht) {
                    mul_f16x2(se[0], ae[0], __shfl_sync(0xffffffffu, f2x[hu], k));
                    mul_f16x2(ew[0], ae[0], __shfl_sync(0xffffffffu, f4[hu], k));
                }
#pragma unroll
                for (int uu = 0; uu < 2; ++uu) {
                    const int u = 2 * hu + uu;
                    const unsigned at = kt + hu * (Cfg::TOK / 2) + b_tok[uu];
                    if (u <= rt) {
                        unsigned be[1][4];
                        ldsm4_t(be[0], at + Cfg::OFF_E);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            mma_pieces<1, 1>(x1[u][n], sy, be, n);
                            mma_pieces<1, 1>(x3[u][n], sw, be, n);
                        }
                    }
                    if (u >= rt) {
                        unsigned by[1][4], bw[1][4];
                        ldsm4_t(by[0], at + Cfg::OFF_Y);
                        ldsm4_t(bw[0], at + Cfg::OFF_W);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            mma_pieces<1, 1>(x2[u][n], se, by, n);
                            if (u == rt) mma_pieces<1, 1>(x4[n], ew, bw, n);
                            else mma_pieces<1, 1>(x3[u][n], ew, bw, n);
                        }
                    }
                }
            }
        }
        // times the decays, beta and the scales taken back out: M1 / ck for dq; M1^T scale / cq
        // and -(M2 + M2^T) / ck for dk
        float m1 = 0.f, m2 = 0.f;
        float grh[2], grl[2], br[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = 16 * rt + g + 8 * r;
            grh[r] = Gh[t]; grl[r] = Gl[t]; br[r] = bet[t];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float e1 = i1[u >> 1] * p.scale * ick[u >> 1], e2 = i2[u >> 1] * p.scale * icq[u >> 1];
            const float e3 = -i3[u >> 1] * ick[u >> 1], e4 = -i4[u >> 1] * ick[u >> 1];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int q0 = 16 * u + 8 * n + 2 * t4;
                const float2 gh = *reinterpret_cast<const float2 *>(Gh + q0), gl = *reinterpret_cast<const float2 *>(Gl + q0);
                const float2 bq = *reinterpret_cast<const float2 *>(bet + q0);
                // f(m, exponent to take, beta of the column): tiles off the diagonal need one side only
                auto each = [&](auto f) {
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        f(m, ((grh[m >> 1] - (m & 1 ? gh.y : gh.x)) + (grl[m >> 1] - (m & 1 ? gl.y : gl.x))) * kLog2e,
                          m & 1 ? bq.y : bq.x);
                };
                if (u < rt) {
                    each([&](int m, float gd, float bc) {
                        const float d = ex2_approx(gd) * bc;
                        x1[u][n][m] *= d * e1;
                        x3[u][n][m] *= d * e3;
                    });
                } else if (u > rt) {
                    each([&](int m, float gd, float) {
                        const float d = ex2_approx(-gd) * br[m >> 1];
                        x2[u][n][m] *= d * e2;
                        x3[u][n][m] *= d * e4;
                    });
                } else {
                    each([&](int m, float gd, float bc) {
                        const int r = g + 8 * (m >> 1), q = 8 * n + 2 * t4 + (m & 1);
                        const float d = ex2_approx(q <= r ? gd : -gd) * (q < r ? bc : br[m >> 1]);       // r(the later, the earlier)
                        x1[u][n][m] = q <= r ? x1[u][n][m] * (d * e1) : 0.f;
                        x2[u][n][m] = q >= r ? x2[u][n][m] * (d * e2) : 0.f;
                        x3[u][n][m] = q < r ? x3[u][n][m] * (d * e3) : q > r ? x4[n][m] * (d * e4) : 0.f;
                    });
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    m1 = fmaxf(m1, fabsf(x1[u][n][m]));
                    m2 = fmaxf(m2, fmaxf(fabsf(x2[u][n][m]), fabsf(x3[u][n][m])));
                }
            }
        }
        const Pow2 c1 = pow2_for(warp_max_bits(m1)), c2 = pow2_for(warp_max_bits(m2));
        unsigned a1[4][1][4], a2[4][1][4], a3[4][1][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            split_tiles<1>(x1[u][0], x1[u][1], c1.c, a1[u]);
            split_tiles<1>(x2[u][0], x2[u][1], c2.c, a2[u]);
            split_tiles<1>(x3[u][0], x3[u][1], c2.c, a3[u]);
        }
        float fq[2], fw[2], fe[2];       // row factors of the products with the states
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = 16 * rt + g + 8 * r;
            fq[r] = p.scale * gam[t] * i5;
            fw[r] = -gam[t] * i6;
            fe[r] = bend[t] * i7;
        }
        // the A operands of the products with the states, at their common scales; kept for all
        // columns where they fit
        constexpr bool HOLD = Cfg::PARTS == 4;
        unsigned hy[HOLD ? 4 : 1][1][4], hw[HOLD ? 4 : 1][1][4], he[HOLD ? 4 : 1][1][4];
        auto load_a = [&](int k, unsigned (&sy)[1][4], unsigned (&sw)[1][4], unsigned (&se)[1][4]) {
            unsigned r[4];
            const unsigned kt = sbase + k * kTok16 + a_tok;
            ldsm4_t(r, kt + Cfg::OFF_Y);
            mul_f16x2(sy[0], r, __shfl_sync(0xffffffffu, f5, k));
            ldsm4_t(r, kt + Cfg::OFF_W);
            mul_f16x2(sw[0], r, __shfl_sync(0xffffffffu, f6, k));
            ldsm4_t(r, kt + Cfg::OFF_E);
            mul_f16x2(se[0], r, __shfl_sync(0xffffffffu, f7, k));
        };
        if constexpr (HOLD)
#pragma unroll
            for (int k = 0; k < 4; ++k) load_a(k, hy[k], hw[k], he[k]);
        // 32 columns at a time
#pragma unroll 1
        for (int j0 = 0; j0 < NP / 32; ++j0) {
            float aq[4][4], ak[4][4], aw[4][4], ae[4][4], am[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) { zero4(aq[n]); zero4(ak[n]); zero4(aw[n]); zero4(ae[n]); zero4(am[n]); }
#pragma unroll 4
            for (int k = 0; k < Cfg::PARTS; ++k) {
                unsigned ty[1][4], tw[1][4], te[1][4];
                if constexpr (!HOLD) load_a(k, ty, tw, te);
                const unsigned (&sy)[1][4] = HOLD ? hy[HOLD ? k : 0] : ty;
                const unsigned (&sw)[1][4] = HOLD ? hw[HOLD ? k : 0] : tw;
                const unsigned (&se)[1][4] = HOLD ? he[HOLD ? k : 0] : te;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    unsigned bS[1][4], bD[1][4];
                    const unsigned at = sbase + k * S16::BYTES + b_st + (unsigned((4 * j0 + 2 * j) * 16) ^ x_st);
                    ldsm4_t(bS[0], at + Cfg::OFF_S);
                    ldsm4_t(bD[0], at + Cfg::OFF_D);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma_pieces<1, 1>(aq[2 * j + n], sy, bS, n);
                        mma_pieces<1, 1>(aw[2 * j + n], sw, bS, n);
                        mma_pieces<1, 1>(ae[2 * j + n], se, bD, n);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    unsigned bK[KP][4], bQ[KP][4];
                    const unsigned at = sbase + Cfg::OFF_KQ + (u >> 1) * Rows::BYTES + (u & 1) * 16 * Rows::ROW + b_kq + j0 * 64 + j * 32;
#pragma unroll
                    for (int i = 0; i < KP; ++i) ldsm4_t(bK[i], at + i * Rows::PIECE);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if (u <= rt) mma_pieces<1, KP>(ak[2 * j + n], a1[u], bK, n);
                        mma_pieces<1, KP>(am[2 * j + n], a3[u], bK, n);
                    }
                    if (u >= rt) {
#pragma unroll
                        for (int i = 0; i < KP; ++i) ldsm4_t(bQ[i], at + (KP + i) * Rows::PIECE);
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_pieces<1, KP>(am[2 * j + n], a2[u], bQ, n);
                    }
                }
            // dq into aq, dk into am; sums over the heads of a key head so far from scratch
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    aq[n][m] = fmaf(c1.inv, ak[n][m], fq[m >> 1] * aq[n][m]);
                    am[n][m] = fmaf(c2.inv, am[n][m], fmaf(fw[m >> 1], aw[n][m], fe[m >> 1] * ae[n][m]));
                }
            if (group > 1) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int t = 16 * rt + g + 8 * r, col = 32 * j0 + 8 * n + 2 * t4;
                        if (t >= nt || col >= p.N) continue;
                        const size_t off = k0 + size_t(t) * krow + col;
                        float2 *pq = reinterpret_cast<float2 *>(p.part + off);
                        float2 *pk = reinterpret_cast<float2 *>(p.part + size_t(p.batch) * p.seqlen * krow + off);
                        float2 q = f2(aq[n][2 * r], aq[n][2 * r + 1]), k = f2(am[n][2 * r], am[n][2 * r + 1]);
                        if (hg > 0) { q = fadd2(*pq, q); k = fadd2(*pk, k); }
                        if (hg + 1 < group) { *pq = q; *pk = k; }
                        aq[n][2 * r] = q.x; aq[n][2 * r + 1] = q.y;
                        am[n][2 * r] = k.x; am[n][2 * r + 1] = k.y;
                    }
            }
            if (hg + 1 == group) {       // 16 rows of 32 columns through the warp's tile: whole 16-byte stores
                unsigned char *tile = smem + Cfg::OFF_OUT + rt * kTok16;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float (&f)[4][4] = x ? am : aq;
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        unsigned r[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) r[m] = pack_bf16x2(f[2 * h2 + (m >> 1)][2 * (m & 1)], f[2 * h2 + (m >> 1)][2 * (m & 1) + 1]);
                        stsm4(smem_u32(tile) + tok16_at(rb, 2 * h2 + (lane >> 4)), r);
                    }
                    __syncwarp();
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int r = 8 * y + (lane >> 2), col = 32 * j0 + 8 * (lane & 3);
                        const uint4 w = *reinterpret_cast<const uint4 *>(tile + tok16_at(r, lane & 3));
                        if (16 * rt + r < nt && col < p.N)
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(x ? p.dk : p.dq) + k0 +
                                                       size_t(16 * rt + r) * krow + col) = w;
                    }
                    __syncwarp();
                }
            }
        }
        if (tid < nt) {
            if (front) for (int x = 0; x < tid; ++x) z -= dtok[x];
            else for (int x = nt - 1; x >= tid; --x) z += dtok[x];
            p.da[gate] = z;
            p.dbeta[gate] = db;
        }
        if (hg + 1 < group) {            // the tiles and vectors are done with
            if (!__syncthreads_and(alive)) { alive = false; break; }
            if (tid == 0) copies(hg + 1);
        }
    }
    if (!alive) {                        // results are void; copies may still be on their way: wait (bounded) for them
        mbar_wait(bar, 0, kDeltaWaitCycles);
        mbar_wait(bar, 1, kDeltaWaitCycles);
    }
}

}  // namespace ssm
