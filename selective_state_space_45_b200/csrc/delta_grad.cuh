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
#pragma once

#include "mma_common.cuh"

namespace ssm {

struct DeltaGradArgs {
    const void *q, *k, *v, *dy;
    const float *a, *beta, *e, *w;
    const float *ck, *dck;             // states and their gradients at the boundaries
    const float *dyy, *edu;            // [slices][batch][heads][seqlen]
    const float *zsum;                 // [zparts][batch][heads][boundaries]
    void *dq, *dk;
    float *da, *dbeta;
    int batch, seqlen, heads, qk_heads, P, N, slices, zparts;
    float scale;
};

constexpr int kGradC = 64, kGradK = 16, kGradPad = 4;

// The decays of a chunk of 64 tokens of one head, from 64-bit prefix sums (a below -1e4
// counts as -1e4: its exponential is 0 either way, and sums stay finite).
struct GradDecay {
    double G[kGradC];
    float gam[kGradC], end[kGradC], beta[kGradC], d[kGradC];
};

template <int NP, typename Tin, typename Tg>
__global__ void __launch_bounds__(256) delta_grad_kernel(const DeltaGradArgs p) {
    constexpr int C = kGradC, KS = kGradK, CT = NP / 64;          // CT: quads of columns per thread
    constexpr int AR = C + kGradPad, BR = NP + kGradPad;
    extern __shared__ __align__(128) unsigned char delta_smem[];
    unsigned char *smem = delta_smem;
    float *A0 = reinterpret_cast<float *>(smem), *A1 = A0 + KS * AR, *A2 = A1 + KS * AR;
    float *B0 = A2 + KS * AR, *B1 = B0 + KS * BR;
    float *M1 = B1 + KS * BR, *M2 = M1 + C * AR;
    GradDecay &dec = *reinterpret_cast<GradDecay *>(M2 + C * AR);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int nchunk = (p.seqlen + C - 1) / C, nbound = nchunk + 1;
    const int c = int(blockIdx.x % unsigned(nchunk)), bk = int(blockIdx.x / unsigned(nchunk));
    const int b = bk / p.qk_heads, hk = bk - b * p.qk_heads;
    const int t0 = c * C, nt = min(C, p.seqlen - t0), group = p.heads / p.qk_heads;
    const size_t krow = size_t(p.qk_heads) * p.N, k0 = (size_t(b) * p.seqlen + t0) * krow + size_t(hk) * p.N;
    const Tin *qp = static_cast<const Tin *>(p.q) + k0, *kp = static_cast<const Tin *>(p.k) + k0;

    // [64 tokens][x0 .. x0 + 16) of rows of `stride` values -> X[column][token], times f(token)
    auto load_t = [&](float *X, const auto *src, size_t stride, int x0, int width, auto f) {
        const int r = tid >> 2, x = (tid & 3) * 4;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < nt && x0 + x < width) {
            loadn<4>(src + size_t(r) * stride + x0 + x, v);
            const float s = f(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= s;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) X[(x + i) * AR + r] = v[i];
    };
    // rows [r0, r0 + 16) of N values -> X[row][column]
    auto load_n = [&](float *X, const auto *src, size_t stride, int r0, int rows) {
        for (int y = tid; y < KS * (NP / 4); y += 256) {
            const int r = y / (NP / 4), n = (y % (NP / 4)) * 4;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (r0 + r < rows && n < p.N) loadn<4>(src + size_t(r0 + r) * stride + n, v);
            *reinterpret_cast<float4 *>(X + r * BR + n) = make_float4(v[0], v[1], v[2], v[3]);
        }
    };
    auto one = [](int) { return 1.f; };
    // acc[i][:] += x[i] * (four columns)
    auto fma4 = [](float2 (&acc)[2], float x, float4 y) {
        acc[0] = ffma2(f2(x, x), f2(y.x, y.y), acc[0]);
        acc[1] = ffma2(f2(x, x), f2(y.z, y.w), acc[1]);
    };
    auto quad = [](const float *x) { return *reinterpret_cast<const float4 *>(x); };

    float2 dq[4][CT][2] = {}, dk[4][CT][2] = {};
    for (int hg = 0; hg < group; ++hg) {
        const int h = hk * group + hg;
        const size_t bh = size_t(b) * p.heads + h, all = size_t(p.batch) * p.heads;
        const size_t vrow = size_t(p.heads) * p.P, v0 = (size_t(b) * p.seqlen + t0) * vrow + size_t(h) * p.P;
        const Tg *dyp = static_cast<const Tg *>(p.dy) + v0;
        const float *ep = p.e + v0, *wp = p.w + v0;
        const float *S0 = p.ck + (bh * nbound + c) * p.P * p.N, *dE = p.dck + (bh * nbound + c + 1) * p.P * p.N;
        // v.w of every token: four threads per token, sixteen bytes of v at a time
        float vw = 0.f;
        {
            const int r = tid >> 2;
            if (r < nt) {
                const Tin *vp = static_cast<const Tin *>(p.v) + v0 + size_t(r) * vrow;
                for (int x = (tid & 3) * 8; x < p.P; x += 32) {
                    float a[8], f[8];
                    load8(vp + x, a);
                    load8(wp + size_t(r) * vrow + x, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) vw = fmaf(a[i], f[i], vw);
                }
            }
            vw += __shfl_xor_sync(0xffffffffu, vw, 1);
            vw += __shfl_xor_sync(0xffffffffu, vw, 2);
        }
        __syncthreads();
        if ((tid & 3) == 0) dec.d[tid >> 2] = vw;
        __syncthreads();
        if (tid < C) {
            const size_t at = (size_t(b) * p.seqlen + t0 + tid) * p.heads + h;
            dec.G[tid] = tid < nt ? double(fmaxf(p.a[at], -1e4f)) : 0.0;
            dec.beta[tid] = tid < nt ? p.beta[at] : 0.f;
            float d = 0.f, db = 0.f;
            if (tid < nt)
                for (int s = 0; s < p.slices; ++s) {
                    const size_t x = (s * all + bh) * p.seqlen + t0 + tid;
                    d += p.dyy[x];
                    db += p.edu[x];
                }
            dec.d[tid] = d - dec.d[tid];
            if (tid < nt) p.dbeta[at] = db;
        }
        __syncthreads();
        double G = 0.0;
        if (tid < C)
            for (int x = 0; x <= tid; ++x) G += dec.G[x];
        __syncthreads();
        if (tid < C) dec.G[tid] = G;
        __syncthreads();
        if (tid < C) {
            dec.gam[tid] = expf(float(G));
            dec.end[tid] = expf(float(dec.G[C - 1] - G));
            if (tid < nt) {
                float z = 0.f;
                const bool front = 2 * tid < nt;
                for (int s = 0; s < p.zparts; ++s) z += p.zsum[(s * all + bh) * nbound + c + (front ? 0 : 1)];
                if (front) for (int x = 0; x < tid; ++x) z -= dec.d[x];
                else for (int x = nt - 1; x >= tid; --x) z += dec.d[x];
                p.da[(size_t(b) * p.seqlen + t0 + tid) * p.heads + h] = z;
            }
        }
        // dy.e and w.e, then M1 and M2
        float2 de[4][2] = {}, we[4][2] = {};
        for (int x0 = 0; x0 < p.P; x0 += KS) {
            __syncthreads();
            load_t(A0, dyp, vrow, x0, p.P, one);
            load_t(A1, wp, vrow, x0, p.P, one);
            load_t(A2, ep, vrow, x0, p.P, one);
            __syncthreads();
#pragma unroll
            for (int x = 0; x < KS; ++x) {
                const float4 da = quad(A0 + x * AR + 4 * ty), wa = quad(A1 + x * AR + 4 * ty), eb = quad(A2 + x * AR + 4 * tx);
                const float d4[4] = {da.x, da.y, da.z, da.w}, w4[4] = {wa.x, wa.y, wa.z, wa.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) { fma4(de[i], d4[i], eb); fma4(we[i], w4[i], eb); }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * ty + i, s = 4 * tx + j;
                const float r = s <= t ? expf(float(dec.G[t] - dec.G[s])) * dec.beta[s] : 0.f;
                M1[t * AR + s] = s <= t ? r * p.scale * (j & 1 ? de[i][j >> 1].y : de[i][j >> 1].x) : 0.f;
                M2[t * AR + s] = s < t ? r * (j & 1 ? we[i][j >> 1].y : we[i][j >> 1].x) : 0.f;
            }
        // the products with the states
        for (int x0 = 0; x0 < p.P; x0 += KS) {
            __syncthreads();
            load_t(A0, dyp, vrow, x0, p.P, [&](int r) { return p.scale * dec.gam[r]; });
            load_t(A1, wp, vrow, x0, p.P, [&](int r) { return -dec.gam[r]; });
            load_t(A2, ep, vrow, x0, p.P, [&](int r) { return dec.beta[r] * dec.end[r]; });
            load_n(B0, S0, p.N, x0, p.P);
            load_n(B1, dE, p.N, x0, p.P);
            __syncthreads();
#pragma unroll 4
            for (int x = 0; x < KS; ++x) {
                const float4 da = quad(A0 + x * AR + 4 * ty), wa = quad(A1 + x * AR + 4 * ty), ea = quad(A2 + x * AR + 4 * ty);
                const float d4[4] = {da.x, da.y, da.z, da.w}, w4[4] = {wa.x, wa.y, wa.z, wa.w}, e4[4] = {ea.x, ea.y, ea.z, ea.w};
#pragma unroll
                for (int m = 0; m < CT; ++m) {
                    const float4 sb = quad(B0 + x * BR + 64 * m + 4 * tx), db = quad(B1 + x * BR + 64 * m + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        fma4(dq[i][m], d4[i], sb);
                        fma4(dk[i][m], w4[i], sb);
                        fma4(dk[i][m], e4[i], db);
                    }
                }
            }
        }
        // the products between the tokens
        for (int s0 = 0; s0 < C; s0 += KS) {
            __syncthreads();
            load_n(B0, qp, krow, s0, nt);
            load_n(B1, kp, krow, s0, nt);
            __syncthreads();
#pragma unroll 4
            for (int x = 0; x < KS; ++x) {
                const float4 m1t = quad(M1 + (s0 + x) * AR + 4 * ty), m2t = quad(M2 + (s0 + x) * AR + 4 * ty);
                const float a1[4] = {m1t.x, m1t.y, m1t.z, m1t.w}, a2[4] = {m2t.x, m2t.y, m2t.z, m2t.w};
#pragma unroll
                for (int m = 0; m < CT; ++m) {
                    const float4 qb = quad(B0 + x * BR + 64 * m + 4 * tx), kb = quad(B1 + x * BR + 64 * m + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        fma4(dq[i][m], M1[(4 * ty + i) * AR + s0 + x], kb);
                        fma4(dk[i][m], a1[i], qb);
                        fma4(dk[i][m], -(a2[i] + M2[(4 * ty + i) * AR + s0 + x]), kb);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 4 * ty + i;
        if (t >= nt) continue;
#pragma unroll
        for (int m = 0; m < CT; ++m) {
            const int n = 64 * m + 4 * tx;
            if (n >= p.N) continue;
            const float xq[4] = {dq[i][m][0].x, dq[i][m][0].y, dq[i][m][1].x, dq[i][m][1].y};
            const float xk[4] = {dk[i][m][0].x, dk[i][m][0].y, dk[i][m][1].x, dk[i][m][1].y};
            storen<4>(static_cast<Tg *>(p.dq) + k0 + size_t(t) * krow + n, xq);
            storen<4>(static_cast<Tg *>(p.dk) + k0 + size_t(t) * krow + n, xk);
        }
    }
}

template <int NP> constexpr int delta_grad_smem() {
    return (3 * kGradK * (kGradC + kGradPad) + 2 * kGradK * (NP + kGradPad) + 2 * kGradC * (kGradC + kGradPad)) * 4 +
           int(sizeof(GradDecay));
}

}  // namespace ssm
