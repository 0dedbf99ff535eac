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
// summed over the value heads that share the key head, in their order.  With
//     X(t,s) = r(t,s) (scale (dy_t.e_s) (q_t.k_s) - [s < t] (w_t.e_s) (k_t.k_s))  for s <= t,
//     F_s = end_s e_s.(dE k_s),   R_t = gam_t (scale dy_t.(S0 q_t) - w_t.(S0 k_t))
// the other two are what passes between the tokens on either side of a decay:
//     dbeta_s = F_s + sum_{t>=s} X(t,s)
//     da_t = sum_{t'>=t} sum_{s<t} X(t',s) beta_s + sum_{t'>=t} R_t' + sum_{s<t} beta_s F_s + gam_last <dE, S0>
// Every term of da_t has the decay exp(a_t) in it, so da_t is as exact beside its own size as the
// products are, and 0 where the decay is.  (<dS, S> at the chunk's end plus the sums of dy.y - v.w
// from there is the same number, but its terms have not: at a = -12 a third of it was rounding.)
//
// Operands.  Every product runs on the tensor cores with scaled fp16 operands, two pieces for
// each value (one for dy, q and k where they come as bf16), as in the passes; the passes leave
// them as tiles of this kernel's shared memory, and bulk copies bring them in: nothing is loaded
// or converted by its threads on the way.  One piece behind bf16 gradients made 13% of them
// round the other way.  A tile's scale is that of its part, 16 rows of headdim, which are one
// step of a product's inner index: before a step its A operand is multiplied with the power of
// two (at most 1) that brings the step's product to the smallest of the parts' scales.
//
// Four warps with 16 tokens (rows) each; where shared memory leaves room for one CTA only, four
// more that take the other half of the state's columns.  The columns go by in slices of 32, the
// next ones on their way as far as the memory reaches.  The token-by-token matrices never leave
// the registers: each is formed in the layout of an accumulator whose rows are the rows it is
// then used with (dy e^T for dq, e dy^T, e w^T and w e^T for dk), so that it becomes the next
// product's A operand as it stands, and tiles off the triangle are skipped; every warp has ten
// of them.  The largest magnitudes that set the scales come from the passes.
//
// What bounds it: latency.  8 x 2048 tokens, 24 heads of 64 x 128, bf16: 597 us, 1.8 TB/s, the
// mma.sync pipe active for 37% of the time; of a warp's cycles 36% go to fixed latencies of
// dependent instructions, 20% to waiting for shared and global memory, 8% to barriers and 8% to
// the pipe, with two warps on a scheduler and no room for more.  3 x 1021 tokens, 8 heads of
// 128 x 64 over 4, fp32: 113 us, 192 CTAs in two rounds.  The compiler spills up to 80
// bytes a thread, most where k and q come in two pieces (none in this bf16 variant).
#pragma once

#include "delta_rule.cuh"

namespace ssm {

struct DeltaGradArgs {
    const float *a, *beta;
    const unsigned char *rows, *prep;  // k and q as operands, and the chunk blocks (their scales)
    const unsigned char *e16, *w16, *y16, *s16, *d16;      // the passes' tiles
    unsigned *timeouts;
    const unsigned *smax, *dsmax;      // [batch][heads][boundaries][zparts]
    const unsigned *emax, *wmax, *ymax;// [batch][heads][chunks of 32][zparts]
    float *part;                       // heads that share a key head: running sums of dq, dk, [2][tokens][qk_heads][N]
    void *dq, *dk;
    float *da, *dbeta;
    int batch, seqlen, heads, qk_heads, P, N, zparts;
    float scale;
};

constexpr int kGradC = 64;                     // tokens per CTA

// NP: dstate padded; PW: headdim padded to 64 or 128; KP: pieces of k and q; Tg: the gradients' type.
template <int NP_, int PW_, int KP_, typename Tg_> struct GradCfg {
    using Tg = Tg_;
    static constexpr int NP = NP_, PW = PW_, KP = KP_, PARTS = PW / 16, PY = sizeof(Tg) == 2 ? 1 : 2;
    using Rows = DeltaRows<NP, KP>;
    static constexpr int TOK = 2 * PARTS * kTok16;         // bytes of a piece of e, w or dy: [half][part][piece]
    static constexpr int OFF_E = 0, OFF_W = 2 * TOK, OFF_Y = 4 * TOK;
    static constexpr int OFF_KQ = OFF_Y + PY * TOK;                           // [half] k and q
    static constexpr int OFF_VEC = OFF_KQ + 2 * Rows::BYTES;
    static constexpr int OFF_OUT = OFF_VEC + 11 * kGradC * 4 + 128;           // X on the diagonal, later the warps' output tiles
    static constexpr int OUT = kTok16;
    static constexpr int SLICE = 4 * PARTS * kTok16;                          // S and dE, 32 columns: [S, dE][part][piece]
    static constexpr int HALF = 113 * 1024, WHOLE = 227 * 1024;               // shared memory for two CTAs on an SM, or one
    static constexpr int fixed(int groups) { return OFF_OUT + 4 * (sizeof(Tg) == 2 ? groups : 1) * OUT; }
    static constexpr int CTAS = fixed(1) + SLICE <= HALF ? 2 : 1;
    static constexpr int NG = CTAS == 2 ? 1 : 2, NT = 128 * NG;               // groups of four warps
    static constexpr int CW = NG == 2 && (NP == 32 || fixed(2) + 2 * SLICE > WHOLE) ? 16 : 32;       // a group's columns in a step
    static constexpr int COLS = NG * CW, SL = COLS / 32, STEPS = (NP + COLS - 1) / COLS;
    static constexpr int ROOM = ((CTAS == 2 ? HALF : WHOLE) - fixed(NG)) / (SL * SLICE);
    static constexpr int STAGES = ROOM < STEPS ? ROOM : STEPS;
    static constexpr int OFF_ST = fixed(NG);
    static constexpr int SMEM_BYTES = OFF_ST + STAGES * SL * SLICE;
    static_assert(STAGES >= 1 && STAGES <= 4);
};

// 2^e as a float and, for e <= 0, as a pair of halves (0 below the smallest).
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(unsigned(min(max(e, -126), 127) + 127) << 23); }
__device__ __forceinline__ unsigned half2_exp2(int e) {
    const __half2 h = __float2half2_rn(exp2_int(e));
    return *reinterpret_cast<const unsigned *>(&h);
}
template <int P> __device__ __forceinline__ void mul_f16x2(unsigned (&o)[P][4], const unsigned (&a)[P][4], unsigned f) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&a[p][i]), *reinterpret_cast<const __half2 *>(&f));
            o[p][i] = *reinterpret_cast<const unsigned *>(&h);
        }
}
// The pieces of a tile, 1 KB apart, as they are or transposed.
template <int P> __device__ __forceinline__ void ldsm4_t_pieces(unsigned (&r)[P][4], unsigned at) {
#pragma unroll
    for (int i = 0; i < P; ++i) ldsm4_t(r[i], at + i * kTok16);
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT, Cfg::CTAS) delta_grad_kernel(const DeltaGradArgs p) {
    using Rows = typename Cfg::Rows;
    using Tg = typename Cfg::Tg;
    constexpr int C = kGradC, NP = Cfg::NP, KP = Cfg::KP, PY = Cfg::PY, PARTS = Cfg::PARTS, NT = Cfg::NT;
    extern __shared__ __align__(128) unsigned char delta_smem[];
    unsigned char *smem = delta_smem;
    // per token: the decays (Gh + Gl the sum of a from the chunk's start, gam its exponential, end that
    // of the rest), beta, 1 / scales of the keys, row sums of X beta left of the diagonal tile, and
    // column sums of X in the tiles of row tile 0..3; then the sums of the tiles left of the diagonal.
    // Gh, Gl, gam and end later hold R and F, a pair for each group of warps, tile those of Z.
    float *Gh = reinterpret_cast<float *>(smem + Cfg::OFF_VEC), *Gl = Gh + C, *gam = Gl + C, *end = gam + C;
    float *bet = end + C, *ick = bet + C, *rowx = ick + C, *colx = rowx + C, *tile = colx + 4 * C;
    double *half = reinterpret_cast<double *>(tile + 16);
    uint64_t *tokbar = reinterpret_cast<uint64_t *>(half + 2), *stbar = tokbar + 1;
    const int tid = threadIdx.x, lane = tid & 31, rt = (tid >> 5) & 3, gr = tid >> 7, ht = rt >> 1, g = lane >> 2, t4 = lane & 3;
    const int nchunk = (p.seqlen + C - 1) / C, nbound = nchunk + 1, nck = (p.seqlen + kDeltaC - 1) / kDeltaC;
    const int c = int(blockIdx.x % unsigned(nchunk)), bk = int(blockIdx.x / unsigned(nchunk));
    const int b = bk / p.qk_heads, hk = bk - b * p.qk_heads;
    const int t0 = c * C, nt = min(C, p.seqlen - t0), group = p.heads / p.qk_heads;
    const int c32 = 2 * c, n32 = min(2, nck - c32), kp = (p.P + 15) / 16;
    const size_t krow = size_t(p.qk_heads) * p.N;
    const size_t k0 = (size_t(b) * p.seqlen + t0) * krow + size_t(hk) * p.N;
    const int total = group * Cfg::STEPS;
    if (tid == 0) {
        mbar_init(tokbar, 1);
        for (int i = 0; i < Cfg::STAGES; ++i) mbar_init(&stbar[i], 1);
        mbar_fence_init();
    }
    auto zero = [&](int off, int bytes) {
        for (int x = tid; x < bytes / 16; x += NT) *reinterpret_cast<uint4 *>(smem + off + 16 * x) = make_uint4(0, 0, 0, 0);
    };
    // a chunk whose second half is past the end: that half is zeros
    if (n32 == 1) {
        zero(Cfg::OFF_E + Cfg::TOK, Cfg::TOK);
        zero(Cfg::OFF_W + Cfg::TOK, Cfg::TOK);
        zero(Cfg::OFF_Y + PY * Cfg::TOK / 2, PY * Cfg::TOK / 2);
        zero(Cfg::OFF_KQ + Rows::BYTES, Rows::BYTES);
    }
    if (kp < PARTS) {                    // parts past headdim: zeros
        const int n = PARTS - kp;
        for (int hf = 0; hf < 2; ++hf) {
            zero(Cfg::OFF_E + hf * Cfg::TOK + kp * 2 * kTok16, n * 2 * kTok16);
            zero(Cfg::OFF_W + hf * Cfg::TOK + kp * 2 * kTok16, n * 2 * kTok16);
            zero(Cfg::OFF_Y + hf * (PY * Cfg::TOK / 2) + kp * PY * kTok16, n * PY * kTok16);
        }
        for (int i = 0; i < 2 * Cfg::SL * Cfg::STAGES; ++i)
            zero(Cfg::OFF_ST + i * (Cfg::SLICE / 2) + kp * 2 * kTok16, n * 2 * kTok16);
    }
    __syncthreads();
    // by one thread: a head's tokens; a step's slices of its states
    auto copy_tokens = [&](int hg) {
        const size_t bh = size_t(b) * p.heads + hk * group + hg;
        const uint32_t tok = kp * kTok16;
        mbar_arrive_expect_tx(tokbar, n32 * ((4 + PY) * tok + (hg == 0 ? Rows::BYTES : 0)));
        for (int hf = 0; hf < n32; ++hf) {
            const size_t at = (bh * nck + c32 + hf) * p.zparts * kTok16;
            bulk_load(smem + Cfg::OFF_E + hf * Cfg::TOK, p.e16 + 2 * at, 2 * tok, tokbar);
            bulk_load(smem + Cfg::OFF_W + hf * Cfg::TOK, p.w16 + 2 * at, 2 * tok, tokbar);
            bulk_load(smem + Cfg::OFF_Y + hf * (PY * Cfg::TOK / 2), p.y16 + PY * at, PY * tok, tokbar);
            if (hg == 0)
                bulk_load(smem + Cfg::OFF_KQ + hf * Rows::BYTES,
                          p.rows + ((size_t(b) * p.qk_heads + hk) * nck + c32 + hf) * Rows::BYTES, Rows::BYTES, tokbar);
        }
    };
    auto copy_states = [&](int it) {
        const int hg = it / Cfg::STEPS, s0 = (it % Cfg::STEPS) * Cfg::SL, ns = min(Cfg::SL, NP / 32 - s0);
        const size_t bh = size_t(b) * p.heads + hk * group + hg;
        const uint32_t bytes = kp * 2 * kTok16;
        unsigned char *to = smem + Cfg::OFF_ST + (it % Cfg::STAGES) * (Cfg::SL * Cfg::SLICE);
        uint64_t *bar = &stbar[it % Cfg::STAGES];
        mbar_arrive_expect_tx(bar, ns * 2 * bytes);
        for (int s = 0; s < ns; ++s) {
            const size_t at = (bh * nbound + c) * (NP / 32) + s0 + s;
            bulk_load(to + s * Cfg::SLICE, p.s16 + at * p.zparts * (2 * kTok16), bytes, bar);
            bulk_load(to + s * Cfg::SLICE + Cfg::SLICE / 2, p.d16 + (at + NP / 32) * p.zparts * (2 * kTok16), bytes, bar);
        }
    };
    if (tid == 0) {
        copy_tokens(0);
        for (int it = 0; it < Cfg::STAGES; ++it) copy_states(it);
    }
    // a bounded wait; after one that gave up the results are void and this thread waits no more
    bool alive = true;
    auto wait = [&](uint64_t *bar, int parity) {
        if (!mbar_test(bar, parity & 1) && alive && !mbar_wait(bar, parity & 1, kDeltaWaitCycles)) {
            alive = false;
            atomicAdd(p.timeouts, 1u);
        }
    };

    // ldmatrix offsets.  e, w, dy tiles are [headdim][token], states [headdim][dstate]: both take
    // the transposing load.  A: this warp's 16 tokens; B: 16 tokens of a half, or 16 columns.
    const int ra = (lane >> 4) * 8 + (lane & 7), rb = (lane >> 3 & 1) * 8 + (lane & 7);
    const unsigned a_tok = tok16_at(ra, (rt & 1) * 2 + (lane >> 3 & 1));
    const unsigned b_tok[2] = {unsigned(tok16_at(rb, lane >> 4)), unsigned(tok16_at(rb, 2 + (lane >> 4)))};
    const unsigned b_kq = b_rows_k(lane, Rows::ROW);
    const unsigned sbase = smem_u32(smem);
    const unsigned aE = sbase + Cfg::OFF_E + ht * Cfg::TOK + a_tok, aW = aE + (Cfg::OFF_W - Cfg::OFF_E);
    const unsigned aY = sbase + Cfg::OFF_Y + ht * (PY * Cfg::TOK / 2) + a_tok;

    auto vec_of = [&](int x) {           // the chunk block's vectors of half x
        return reinterpret_cast<const float *>(p.prep + ((size_t(b) * p.heads + hk * group) * nck + c32 + (x < n32 ? x : 0)) *
                                                            DeltaBlock::BYTES + DeltaBlock::OFF_VEC);
    };
    float icq[2];                        // 1 / scales of q in the chunk's halves
#pragma unroll
    for (int x = 0; x < 2; ++x) icq[x] = __ldg(vec_of(x) + kVecScalars * kDeltaC + kInvQ);
    if (tid < C) ick[tid] = __ldg(vec_of(tid >> 5) + kVecL * kDeltaC + (tid & 31)) * (1.f / 8192.f);
    const unsigned own = sbase + Cfg::OFF_KQ + ht * Rows::BYTES;         // the half's k and q, and the warp's rows of them
    const unsigned a_kq = own + ((rt & 1) * 16 + (lane & 15)) * Rows::ROW + (lane >> 4) * 16, n_kq = b_rows_n(lane, Rows::ROW);
    bool dead = false;
    for (int hg = 0; hg < group && !dead; ++hg) {
        const int h = hk * group + hg;
        const size_t bh = size_t(b) * p.heads + h;
        // Everything small at once: scales, and for threads 0..63 their token's gates and sums.
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
        float av = 0.f, bv = 0.f, last = 0.f;
        if (tid < nt) {
            av = __ldg(p.a + gate);
            av = av < -1e4f ? -1e4f : av;                 // (fmaxf would drop a NaN)
            bv = __ldg(p.beta + gate);
        }
        // Scales as powers of two: per product the smallest over the parts (the products come out
        // times 2^it) and each part's distance to it.
        int ly[2], le[2], lw[2];
        constexpr int kBad = -(1 << 16);                  // of a part with an infinite value
        auto log_scale = [&](unsigned m) { return m >= 0x7f800000u ? kBad : int(__float_as_uint(pow2_for(m).c) >> 23) - 127; };
#pragma unroll
        for (int x = 0; x < 2; ++x) { ly[x] = log_scale(bits[x]); le[x] = log_scale(bits[2 + x]); lw[x] = log_scale(bits[4 + x]); }
        const int ls = log_scale(bits[6]), ld = log_scale(bits[7]);
        auto common = [&](int l, float &inv) {
            const int least = __reduce_min_sync(0xffffffffu, lane < kp ? l : 1 << 20);
            inv = exp2_int(-(least >> 1)) * exp2_int((least >> 1) - least);       // 0 when too small for a float
            if (least < kBad / 2) inv = __uint_as_float(kNanBits);
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
            end[tid] = expf(float(Gend - G));
            bet[tid] = bv;
            last = expf(float(Gend));
        }
        __syncthreads();
        wait(tokbar, hg);

        // The token-by-token matrices of this warp's rows, in four tiles of 16 columns: dy e^T;
        // e dy^T; w e^T up to the diagonal and e w^T past it; e w^T on it.
        float x1[4][2][4], x2[4][2][4], x3[4][2][4], x4[2][4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < 2; ++n) { zero4(x1[u][n]); zero4(x2[u][n]); zero4(x3[u][n]); }
        zero4(x4[0]); zero4(x4[1]);
#pragma unroll 2
        for (int k = 0; k < PARTS; ++k) {
            unsigned ay[PY][4], ae[2][4], aw[2][4];
            ldsm4_t_pieces(ay, aY + k * (PY * kTok16));
            ldsm4_t_pieces(ae, aE + k * (2 * kTok16));
            ldsm4_t_pieces(aw, aW + k * (2 * kTok16));
#pragma unroll
            for (int hu = 0; hu < 2; ++hu) {
                unsigned sy[PY][4], se[2][4], sw[2][4], ew[2][4];
                if (hu <= ht) {
                    mul_f16x2(sy, ay, __shfl_sync(0xffffffffu, f1[hu], k));
                    mul_f16x2(sw, aw, __shfl_sync(0xffffffffu, f3[hu], k));
                }
                if (hu >= ht) {
                    mul_f16x2(se, ae, __shfl_sync(0xffffffffu, f2x[hu], k));
                    mul_f16x2(ew, ae, __shfl_sync(0xffffffffu, f4[hu], k));
                }
                const unsigned bE = sbase + Cfg::OFF_E + hu * Cfg::TOK + k * (2 * kTok16), bW = bE + (Cfg::OFF_W - Cfg::OFF_E);
                const unsigned bY = sbase + Cfg::OFF_Y + hu * (PY * Cfg::TOK / 2) + k * (PY * kTok16);
#pragma unroll
                for (int uu = 0; uu < 2; ++uu) {
                    const int u = 2 * hu + uu;
                    if (u <= rt) {
                        unsigned be[2][4];
                        ldsm4_t_pieces(be, bE + b_tok[uu]);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            mma_pieces<PY, 2>(x1[u][n], sy, be, n);
                            mma_pieces<2, 2>(x3[u][n], sw, be, n);
                        }
                    }
                    if (u >= rt) {
                        unsigned by[PY][4], bw[2][4];
                        ldsm4_t_pieces(by, bY + b_tok[uu]);
                        ldsm4_t_pieces(bw, bW + b_tok[uu]);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            mma_pieces<2, PY>(x2[u][n], se, by, n);
                            if (u == rt) mma_pieces<2, 2>(x4[n], ew, bw, n);
                            else mma_pieces<2, 2>(x3[u][n], ew, bw, n);
                        }
                    }
                }
            }
        }
        // times the decays, beta and the scales taken back out: M1 / ck for dq; M1^T scale / cq
        // and -(M2 + M2^T) / ck for dk; and X up to the diagonal, its sums (one group of warps)
        float m1 = 0.f, m2 = 0.f, rowsum[2] = {0.f, 0.f};
        float grh[2], grl[2], br[2], kr[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = 16 * rt + g + 8 * r;
            grh[r] = Gh[t]; grl[r] = Gl[t]; br[r] = bet[t]; kr[r] = ick[t];
        }
        float *diag = reinterpret_cast<float *>(smem + Cfg::OFF_OUT);
        auto diag_at = [&](int tl, int r, int q) { return tl * 256 + r * 16 + (q ^ r); };       // rows' values in other banks
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float qk[2][4], kk[2][4], xe[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) { zero4(qk[n]); zero4(kk[n]); zero4(xe[n]); }
            if (gr == 0 && u <= rt) {        // q.k and k.k of the tile
#pragma unroll 2
                for (int j = 0; j < NP / 16; ++j) {
                    unsigned ak[KP][4], aq[KP][4], bK[KP][4];
                    const unsigned at = sbase + Cfg::OFF_KQ + (u >> 1) * Rows::BYTES + (u & 1) * 16 * Rows::ROW + n_kq + j * 32;
#pragma unroll
                    for (int x = 0; x < KP; ++x) {
                        ldsm4(ak[x], a_kq + x * Rows::PIECE + j * 32);
                        ldsm4(aq[x], a_kq + (KP + x) * Rows::PIECE + j * 32);
                        ldsm4(bK[x], at + x * Rows::PIECE);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma_pieces<KP, KP>(qk[n], aq, bK, n);
                        mma_pieces<KP, KP>(kk[n], ak, bK, n);
                    }
                }
            }
            const float e1 = i1[u >> 1] * p.scale, e2 = i2[u >> 1] * p.scale * icq[u >> 1];
            const float e3 = -i3[u >> 1], e4 = -i4[u >> 1];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int q0 = 16 * u + 8 * n + 2 * t4;
                const float2 gh = *reinterpret_cast<const float2 *>(Gh + q0), gl = *reinterpret_cast<const float2 *>(Gl + q0);
                const float2 bq = *reinterpret_cast<const float2 *>(bet + q0), kq = *reinterpret_cast<const float2 *>(ick + q0);
                // f(m, exponent to take, beta of the column, 1 / its key's scale): tiles off the diagonal need one side only
                auto each = [&](auto f) {
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        f(m, ((grh[m >> 1] - (m & 1 ? gh.y : gh.x)) + (grl[m >> 1] - (m & 1 ? gl.y : gl.x))) * kLog2e,
                          m & 1 ? bq.y : bq.x, m & 1 ? kq.y : kq.x);
                };
                // a value of X from those of M1 and M2 over beta
                auto pair = [&](int m, float v1, float v3) {
                    xe[n][m] = fmaf(v1, qk[n][m] * icq[ht], v3 * (kk[n][m] * kr[m >> 1]));
                };
                if (u < rt) {
                    each([&](int m, float gd, float bc, float kc) {
                        const float d = ex2_approx(gd) * kc;
                        const float v1 = x1[u][n][m] * (d * e1), v3 = x3[u][n][m] * (d * e3);
                        pair(m, v1, v3);
                        x1[u][n][m] = v1 * bc;
                        x3[u][n][m] = v3 * bc;
                        rowsum[m >> 1] = fmaf(xe[n][m], bc, rowsum[m >> 1]);
                    });
                } else if (u > rt) {
                    each([&](int m, float gd, float, float kc) {
                        const float d = ex2_approx(-gd) * br[m >> 1];
                        x2[u][n][m] *= d * e2;
                        x3[u][n][m] *= d * kc * e4;
                    });
                } else {
                    each([&](int m, float gd, float bc, float kc) {
                        const int r = g + 8 * (m >> 1), q = 8 * n + 2 * t4 + (m & 1);
                        const float d = ex2_approx(q <= r ? gd : -gd), dk = d * kc;       // r(the later, the earlier)
                        const float v1 = q <= r ? x1[u][n][m] * (dk * e1) : 0.f, v3 = q < r ? x3[u][n][m] * (dk * e3) : 0.f;
                        pair(m, v1, v3);
                        x1[u][n][m] = v1 * bc;
                        x2[u][n][m] = q >= r ? x2[u][n][m] * (d * br[m >> 1] * e2) : 0.f;
                        x3[u][n][m] = q < r ? v3 * bc : q > r ? x4[n][m] * (dk * br[m >> 1] * e4) : 0.f;
                        if (gr == 0) diag[diag_at(rt, r, q)] = xe[n][m] * bc;
                    });
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    m1 = fmaxf(m1, fabsf(x1[u][n][m]));
                    m2 = fmaxf(m2, fmaxf(fabsf(x2[u][n][m]), fabsf(x3[u][n][m])));
                }
            }
            if (gr == 0 && u <= rt) {        // the tile's column sums, and its own
                float whole = 0.f;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float s = xe[n][y] + xe[n][y + 2];
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                        const int q = 16 * u + 8 * n + 2 * t4 + y;
                        if (g == 0) colx[rt * C + q] = s;
                        whole = fmaf(s, bet[q], whole);
                    }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) whole += __shfl_xor_sync(0xffffffffu, whole, o);
                if (lane == 0) tile[4 * rt + u] = whole;
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) rowsum[r] += __shfl_xor_sync(0xffffffffu, rowsum[r], o);
            if (gr == 0 && t4 == 0) rowx[16 * rt + g + 8 * r] = rowsum[r];
        }
        const Pow2 c1 = pow2_for(warp_max_bits(m1)), c2 = pow2_for(warp_max_bits(m2));
        unsigned a1[4][2][4], a2[4][2][4], a3[4][2][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            split_tiles<2>(x1[u][0], x1[u][1], c1.c, a1[u]);
            split_tiles<2>(x2[u][0], x2[u][1], c2.c, a2[u]);
            split_tiles<2>(x3[u][0], x3[u][1], c2.c, a3[u]);
        }
        float fq[2], fw[2], fe[2];       // row factors of the products with the states
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = 16 * rt + g + 8 * r;
            fq[r] = p.scale * gam[t] * i5;
            fw[r] = -gam[t] * i6;
            fe[r] = end[t] * i7;
        }
        __syncthreads();
        // thread t: the pairs on either side of token t's decay, by tiles (both beside t's; one in it; in
        // the diagonal tile by its rows' running sums), and the column t
        float da = 0.f, db = 0.f;
        if (tid < C) {
            const int tl = tid >> 4, i = tid & 15;
            float run = 0.f;
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                run += diag[diag_at(tl, i, q)];
                diag[diag_at(tl, i, q)] = run;
            }
            __syncwarp();
            for (int r = i; r < 16; ++r) da += rowx[16 * tl + r] + (i > 0 ? diag[diag_at(tl, r, i - 1)] : 0.f);
            for (int m = tl; m < 4; ++m) {
                db += colx[m * C + tid];
                if (m > tl) {
                    for (int q = 0; q < i; ++q) da = fmaf(bet[16 * tl + q], colx[m * C + 16 * tl + q], da);
                    for (int n = 0; n < tl; ++n) da += tile[4 * m + n];
                }
            }
        }
        __syncthreads();
        float rq[2] = {0.f, 0.f}, rk[2] = {0.f, 0.f}, ek[2] = {0.f, 0.f}, z = 0.f;       // parts of R, of F and of Z = <dE, S0>
        // CW columns a step and group
        constexpr int NJ = Cfg::CW / 16;
#pragma unroll 1
        for (int i = 0; i < Cfg::STEPS; ++i) {
            const int it = hg * Cfg::STEPS + i, col0 = i * Cfg::COLS + gr * Cfg::CW;
            wait(&stbar[it % Cfg::STAGES], it / Cfg::STAGES);
            const unsigned char *slices = smem + Cfg::OFF_ST + (it % Cfg::STAGES) * (Cfg::SL * Cfg::SLICE);
            for (int x = tid; x < min(Cfg::SL, NP / 32 - i * Cfg::SL) * PARTS * 64; x += NT) {      // <dE, S0>, 16 bytes a turn
                const int k = (x >> 6) % PARTS;           // the same for a warp
                const unsigned char *at = slices + x / (64 * PARTS) * Cfg::SLICE + k * (2 * kTok16) + (x & 63) * 16;
                uint4 w[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) w[y] = *reinterpret_cast<const uint4 *>(at + (y >> 1) * (Cfg::SLICE / 2) + (y & 1) * kTok16);
                auto value = [&](int m, int y) {
                    auto h = [&](const uint4 &v) { return __half22float2(*(reinterpret_cast<const __half2 *>(&v) + y)); };
                    return fadd2(h(w[2 * m]), h(w[2 * m + 1]));
                };
                float2 s = f2(0.f, 0.f);
#pragma unroll
                for (int y = 0; y < 4; ++y) s = ffma2(value(0, y), value(1, y), s);
                const int l = __shfl_sync(0xffffffffu, ls, k) + __shfl_sync(0xffffffffu, ld, k);
                z += l < kBad / 2 ? __uint_as_float(kNanBits) : (s.x + s.y) * exp2_int(-(l >> 1)) * exp2_int((l >> 1) - l);
            }
            if (col0 < NP) {
                float aq[2 * NJ][4], am[2 * NJ][4];       // dq, dk
                {
                    // the products with the states
                    const unsigned st = smem_u32(slices) + (gr * Cfg::CW / 32) * Cfg::SLICE;
                    const int piece0 = (gr * Cfg::CW % 32) / 8;
                    float aw[2 * NJ][4], ae[2 * NJ][4];
#pragma unroll
                    for (int n = 0; n < 2 * NJ; ++n) { zero4(aq[n]); zero4(aw[n]); zero4(ae[n]); }
#pragma unroll 2
                    for (int k = 0; k < PARTS; ++k) {
                        unsigned sy[PY][4], sw[2][4], se[2][4];
                        ldsm4_t_pieces(sy, aY + k * (PY * kTok16));
                        mul_f16x2(sy, sy, __shfl_sync(0xffffffffu, f5, k));
                        ldsm4_t_pieces(sw, aW + k * (2 * kTok16));
                        mul_f16x2(sw, sw, __shfl_sync(0xffffffffu, f6, k));
                        ldsm4_t_pieces(se, aE + k * (2 * kTok16));
                        mul_f16x2(se, se, __shfl_sync(0xffffffffu, f7, k));
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            unsigned bS[2][4], bD[2][4];
                            const unsigned at = st + k * (2 * kTok16) + tok16_at(rb, piece0 + 2 * j + (lane >> 4));
                            ldsm4_t_pieces(bS, at);
                            ldsm4_t_pieces(bD, at + Cfg::SLICE / 2);
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                mma_pieces<PY, 2>(aq[2 * j + n], sy, bS, n);
                                mma_pieces<2, 2>(aw[2 * j + n], sw, bS, n);
                                mma_pieces<2, 2>(ae[2 * j + n], se, bD, n);
                            }
                        }
                    }
                    // row by row with the token's own q and k: R and F
#pragma unroll
                    for (int n = 0; n < 2 * NJ; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const unsigned char *at = smem + Cfg::OFF_KQ + ht * Rows::BYTES + ((rt & 1) * 16 + g + 8 * r) * Rows::ROW +
                                                      (col0 + 8 * n + 2 * t4) * 2;
                            float2 k = f2(0.f, 0.f), q = f2(0.f, 0.f);
#pragma unroll
                            for (int x = 0; x < KP; ++x) {
                                k = fadd2(k, __half22float2(*reinterpret_cast<const __half2 *>(at + x * Rows::PIECE)));
                                q = fadd2(q, __half22float2(*reinterpret_cast<const __half2 *>(at + (KP + x) * Rows::PIECE)));
                            }
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int m = 2 * r + y;
                                aq[n][m] *= fq[r];
                                aw[n][m] *= fw[r];
                                ae[n][m] *= fe[r];
                                rq[r] = fmaf(aq[n][m], y ? q.y : q.x, rq[r]);
                                rk[r] = fmaf(aw[n][m], y ? k.y : k.x, rk[r]);
                                ek[r] = fmaf(ae[n][m], y ? k.y : k.x, ek[r]);
                                am[n][m] = fmaf(br[r], ae[n][m], aw[n][m]);
                            }
                        }
                }
                // and with the other tokens' k and q
                float bq[2 * NJ][4], bm[2 * NJ][4];
#pragma unroll
                for (int n = 0; n < 2 * NJ; ++n) { zero4(bq[n]); zero4(bm[n]); }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        unsigned bK[KP][4], bQ[KP][4];
                        const unsigned at = sbase + Cfg::OFF_KQ + (u >> 1) * Rows::BYTES + (u & 1) * 16 * Rows::ROW + b_kq + col0 * 2 + j * 32;
#pragma unroll
                        for (int x = 0; x < KP; ++x) ldsm4_t(bK[x], at + x * Rows::PIECE);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            if (u <= rt) mma_pieces<2, KP>(bq[2 * j + n], a1[u], bK, n);
                            mma_pieces<2, KP>(bm[2 * j + n], a3[u], bK, n);
                        }
                        if (u >= rt) {
#pragma unroll
                            for (int x = 0; x < KP; ++x) ldsm4_t(bQ[x], at + (KP + x) * Rows::PIECE);
#pragma unroll
                            for (int n = 0; n < 2; ++n) mma_pieces<2, KP>(bm[2 * j + n], a2[u], bQ, n);
                        }
                    }
#pragma unroll
                for (int n = 0; n < 2 * NJ; ++n)
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        aq[n][m] = fmaf(c1.inv, bq[n][m], aq[n][m]);
                        am[n][m] = fmaf(c2.inv, bm[n][m], am[n][m]);
                    }
                // sums over the heads of a key head so far from scratch; fp32 gradients straight out
                if (group > 1 || sizeof(Tg) == 4) {
#pragma unroll
                    for (int n = 0; n < 2 * NJ; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int t = 16 * rt + g + 8 * r, col = col0 + 8 * n + 2 * t4;
                            if (t >= nt || col >= p.N) continue;
                            const size_t off = k0 + size_t(t) * krow + col;
                            float2 *pq = reinterpret_cast<float2 *>(p.part + off);
                            float2 *pk = reinterpret_cast<float2 *>(p.part + size_t(p.batch) * p.seqlen * krow + off);
                            float2 q = f2(aq[n][2 * r], aq[n][2 * r + 1]), k = f2(am[n][2 * r], am[n][2 * r + 1]);
                            if (hg > 0) { q = fadd2(*pq, q); k = fadd2(*pk, k); }
                            if (hg + 1 < group) {
                                *pq = q; *pk = k;
                            } else if constexpr (sizeof(Tg) == 4) {
                                *reinterpret_cast<float2 *>(static_cast<float *>(p.dq) + off) = q;
                                *reinterpret_cast<float2 *>(static_cast<float *>(p.dk) + off) = k;
                            }
                            aq[n][2 * r] = q.x; aq[n][2 * r + 1] = q.y;
                            am[n][2 * r] = k.x; am[n][2 * r + 1] = k.y;
                        }
                }
                if constexpr (sizeof(Tg) == 2)
                    if (hg + 1 == group) {       // 16 rows through the warp's tile: whole 16-byte stores
                        unsigned char *to = smem + Cfg::OFF_OUT + (tid >> 5) * Cfg::OUT;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float (&f)[2 * NJ][4] = x ? am : aq;
#pragma unroll
                            for (int h2 = 0; h2 < NJ; ++h2) {
                                unsigned r[4];
#pragma unroll
                                for (int m = 0; m < 4; ++m) r[m] = pack_bf16x2(f[2 * h2 + (m >> 1)][2 * (m & 1)], f[2 * h2 + (m >> 1)][2 * (m & 1) + 1]);
                                stsm4(smem_u32(to) + tok16_at(rb, 2 * h2 + (lane >> 4)), r);
                            }
                            __syncwarp();
#pragma unroll
                            for (int y = 0; y < NJ; ++y) {
                                const int r = (16 / NJ) * y + lane / (2 * NJ), pc = lane % (2 * NJ), col = col0 + 8 * pc;
                                const uint4 w = *reinterpret_cast<const uint4 *>(to + tok16_at(r, pc));
                                if (16 * rt + r < nt && col < p.N)
                                    *reinterpret_cast<uint4 *>(static_cast<Tg *>(x ? p.dk : p.dq) + k0 + size_t(16 * rt + r) * krow + col) = w;
                            }
                            __syncwarp();
                        }
                    }
            }
            const bool more = it + Cfg::STAGES < total, next = i + 1 == Cfg::STEPS && hg + 1 < group;
            if (more || next) {              // this step's memory (at a head's end its tokens' too) is done with
                if (!__syncthreads_and(alive)) { alive = false; dead = true; break; }
                if (tid == 0) {
                    if (next) copy_tokens(hg + 1);
                    if (more) copy_states(it + Cfg::STAGES);
                }
            }
        }
        if (dead) break;
        // the head's da and dbeta
        float *R = gr ? gam : Gh, *F = gr ? end : Gl;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            rq[r] = fmaf(rq[r], icq[ht], rk[r] * kr[r]);
            ek[r] *= kr[r];
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                rq[r] += __shfl_xor_sync(0xffffffffu, rq[r], o);
                ek[r] += __shfl_xor_sync(0xffffffffu, ek[r], o);
            }
            if (t4 == 0) {
                R[16 * rt + g + 8 * r] = rq[r];
                F[16 * rt + g + 8 * r] = ek[r];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) tile[tid >> 5] = z;
        __syncthreads();
        if (tid < nt) {
            z = 0.f;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) z += tile[w];
            for (int x = 0; x < nt; ++x) {
                const float f = Gl[x] + (Cfg::NG == 2 ? end[x] : 0.f), r = Gh[x] + (Cfg::NG == 2 ? gam[x] : 0.f);
                da += x < tid ? bet[x] * f : r;
                if (x == tid) db += f;
            }
            p.da[gate] = fmaf(last, z, da);
            p.dbeta[gate] = db;
        }
        if (hg + 1 < group) __syncthreads();
    }
    if (!alive)                          // results are void; copies may still be on their way: wait (bounded) for them
        for (int x = 0; x < 2; ++x) {
            mbar_wait(tokbar, x, kDeltaWaitCycles);
            for (int i = 0; i < Cfg::STAGES; ++i) mbar_wait(&stbar[i], x, kDeltaWaitCycles);
        }
}

}  // namespace ssm
