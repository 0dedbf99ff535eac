// delta_step.cuh -- decode tokens of the gated delta rule, the state updated in place.
//
// Per row of the state (one value of headdim) and token:
//     S' = exp(a) S,  e = v - S'.k,  S = S' + beta e k,  y = scale S.q = scale (S'.q + beta e k.q)
// The last form takes both inner products of a row in one pass over it, so the reductions of
// a token are one round of shuffles.  Bound by HBM: the fp32 state in and out (8 bytes an
// element) against a few hundred bytes per token and head.
//
// Eight lanes share a row and hold dstate / 8 of it as 16-byte quads 128 bytes apart (each
// load of a warp covers four rows' 128-byte lines); a warp takes 8 rows of one head, two
// per lane group, so a head's k and q are read once for both.  The state stays in registers
// through the call's tokens.  256 sequences x 24 heads of 64 x 128, one token: 75 us for 403 MB
// in and out, 83% of HBM's copy rate; one sequence of 16 heads of 128 x 128, four tokens:
// 6.6 us, launch and latency.
#pragma once

#include "common.cuh"

namespace ssm {

struct DeltaStepArgs {
    float *state;             // [batch][heads][P][N]
    const void *q, *k;        // [ntok][batch][qk_heads][N]
    const void *v;            // [ntok][batch][heads][P]
    const float *a, *beta;    // [ntok][batch][heads]
    void *y;                  // [ntok][batch][heads][P]
    int ntok, batch, heads, qk_heads, P, N;
    float scale;
};

template <int Q, typename Tin, typename Tout>        // Q: quads of a row per lane, 32 Q >= N
__global__ void __launch_bounds__(256) delta_step_kernel(const DeltaStepArgs p) {
    constexpr int R = 2;                              // rows per group of eight lanes
    const long long warps = (long long)p.batch * p.heads * (p.P / 8);
    const long long wid = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (wid >= warps) return;
    const int lane = threadIdx.x & 31, l = lane & 7, g = lane >> 3;
    const long long bh = wid / (p.P / 8);
    const int row0 = int(wid - bh * (p.P / 8)) * 8 + g, b = int(bh / p.heads), h = int(bh - (long long)b * p.heads);
    const int hk = h / (p.heads / p.qk_heads);
    float *sp = p.state + (size_t(bh) * p.P + row0) * p.N + 4 * l;
    float4 s[R][Q];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < Q; ++i)
            s[r][i] = 32 * i + 4 * l < p.N ? *reinterpret_cast<const float4 *>(sp + size_t(4 * r) * p.N + 32 * i)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = 0; t < p.ntok; ++t) {
        const size_t tb = size_t(t) * p.batch + b, koff = (tb * p.qk_heads + hk) * p.N + 4 * l;
        const Tin *kp = static_cast<const Tin *>(p.k) + koff, *qp = static_cast<const Tin *>(p.q) + koff;
        const size_t voff = (tb * p.heads + h) * p.P + row0;
        float k[Q][4], q[Q][4], v[R];
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            if (32 * i + 4 * l < p.N) {
                loadn<4>(kp + 32 * i, k[i]);
                loadn<4>(qp + 32 * i, q[i]);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) k[i][x] = q[i][x] = 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = to_f32(static_cast<const Tin *>(p.v)[voff + 4 * r]);
        const float alpha = expf(p.a[tb * p.heads + h]), beta = p.beta[tb * p.heads + h];
        float dk[R], dq[R], kq = 0.f;
#pragma unroll
        for (int i = 0; i < Q; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) kq = fmaf(k[i][x], q[i][x], kq);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 ak = f2(0.f, 0.f), aq = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float2 lo = fmul2(f2(alpha, alpha), f2(s[r][i].x, s[r][i].y));
                const float2 hi = fmul2(f2(alpha, alpha), f2(s[r][i].z, s[r][i].w));
                s[r][i] = make_float4(lo.x, lo.y, hi.x, hi.y);
                ak = ffma2(lo, f2(k[i][0], k[i][1]), ak);
                ak = ffma2(hi, f2(k[i][2], k[i][3]), ak);
                aq = ffma2(lo, f2(q[i][0], q[i][1]), aq);
                aq = ffma2(hi, f2(q[i][2], q[i][3]), aq);
            }
            dk[r] = ak.x + ak.y;
            dq[r] = aq.x + aq.y;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            kq += __shfl_xor_sync(0xffffffffu, kq, o);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                dk[r] += __shfl_xor_sync(0xffffffffu, dk[r], o);
                dq[r] += __shfl_xor_sync(0xffffffffu, dq[r], o);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float u = beta * (v[r] - dk[r]);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                s[r][i].x = fmaf(u, k[i][0], s[r][i].x);
                s[r][i].y = fmaf(u, k[i][1], s[r][i].y);
                s[r][i].z = fmaf(u, k[i][2], s[r][i].z);
                s[r][i].w = fmaf(u, k[i][3], s[r][i].w);
            }
            if (l == 0) static_cast<Tout *>(p.y)[voff + 4 * r] = from_f32<Tout>(p.scale * fmaf(u, kq, dq[r]));
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < Q; ++i)
            if (32 * i + 4 * l < p.N) *reinterpret_cast<float4 *>(sp + size_t(4 * r) * p.N + 32 * i) = s[r][i];
}

}  // namespace ssm
