// delta_bwd_api.cu -- C ABI of the gated delta rule's backward (ssm_delta_rule_bwd): the
// forward pass again (e and the states every 64 tokens), the reverse pass (dv, the state's
// gradient at the same places), then the chunks' gradients in parallel.  Long sequences of few
// heads go through the two passes in segments that run at once, as in the forward.  Scratch: the
// caller's workspace or a stream-ordered buffer.
#include "delta_grad.cuh"
#include "delta_host.cuh"

using namespace ssm_host;

namespace {

template <int NP, int PW, typename Tin, typename Tg> int launch_grad(const ssm::DeltaGradArgs &a, cudaStream_t s) {
    const long long ctas = (long long)a.batch * a.qk_heads * ((a.seqlen + ssm::kGradC - 1) / ssm::kGradC);
    if (ctas > INT_MAX) return SSM_ERR_UNSUPPORTED;
    using Cfg = ssm::GradCfg<NP, PW, (sizeof(Tin) == 4 ? 2 : 1), Tg>;
    if (const int st = set_smem(ssm::delta_grad_kernel<Cfg>, Cfg::SMEM_BYTES)) return st;
    ssm::delta_grad_kernel<Cfg><<<unsigned(ctas), Cfg::NT, Cfg::SMEM_BYTES, s>>>(a);
    return status_of(cudaGetLastError());
}
template <int PW, typename Tin, typename Tg> int dispatch_grad(const ssm::DeltaGradArgs &a, cudaStream_t s) {
    switch (padded_state(a.N)) {
    case 32: return launch_grad<32, PW, Tin, Tg>(a, s);
    case 64: return launch_grad<64, PW, Tin, Tg>(a, s);
    case 96: return launch_grad<96, PW, Tin, Tg>(a, s);
    default: return launch_grad<128, PW, Tin, Tg>(a, s);
    }
}

// The parts of a call's scratch, in this order; each starts on 16 bytes.
struct BwdParts {
    size_t prep, rows, e16, w16, y16, s16, d16, smax, dsmax, emax, wmax, ymax, part, seg_state, seg_map, all;
    int nseg;
    BwdParts(int batch, int seqlen, int heads, int qk_heads, int P, int N, int in_dtype, int grad_dtype) {
        const size_t bh = size_t(batch) * heads;
        const size_t nbound = (size_t(seqlen) + ssm::kDeltaSave - 1) / ssm::kDeltaSave + 1;
        const size_t parts = size_t(delta_slices(P)) * kDeltaWarps;       // of 16 rows
        const size_t state = bh * nbound * parts * 16 * padded_state(N) * 4;
        const size_t tok16 = bh * delta_chunks(seqlen) * parts * ssm::kTok16;       // a piece of e, w or dy
        size_t at = 0;
        auto add = [&](size_t &where, size_t bytes) { where = at; at += round16(bytes); };
        add(prep, prep_bytes(batch, seqlen, heads));
        add(rows, rows_bytes(batch, seqlen, qk_heads, N, in_dtype));
        add(e16, 2 * tok16);
        add(w16, 2 * tok16);
        add(y16, grad_dtype == SSM_BF16 ? tok16 : 2 * tok16);
        add(s16, state);
        add(d16, state);
        add(smax, 4 * parts * bh * nbound);
        add(dsmax, 4 * parts * bh * nbound);
        add(emax, 4 * parts * bh * delta_chunks(seqlen));
        add(wmax, 4 * parts * bh * delta_chunks(seqlen));
        add(ymax, 4 * parts * bh * delta_chunks(seqlen));
        add(part, heads > qk_heads ? 2 * size_t(batch) * seqlen * qk_heads * N * 4 : 0);
        nseg = segments(batch, seqlen, heads, P, N, in_dtype == SSM_F32 || grad_dtype == SSM_F32, true);
        add(seg_state, nseg > 1 ? bh * nseg * P * N * 4 : 0);
        add(seg_map, nseg > 1 ? bh * nseg * N * N * 4 : 0);
        all = at;
    }
};

template <typename T> constexpr int code_of() { return sizeof(T) == 4 ? SSM_F32 : SSM_BF16; }

template <typename Tin, typename Tg>
int run_bwd(ssm::DeltaArgs f, const void *v, const void *dy, const float *dfinal, void *dq, void *dk, void *dv, float *da,
            float *dbeta, float *dh0, void *workspace, size_t bytes, cudaStream_t s) {
    const BwdParts at(f.batch, f.seqlen, f.heads, f.qk_heads, f.P, f.N, code_of<Tin>(), code_of<Tg>());
    Scratch ws;
    if (const int st = ws.take(workspace, bytes, at.all, s)) return st;
    auto part = [&](size_t off) { return reinterpret_cast<float *>(ws.p + off); };
    constexpr int KP = sizeof(Tin) == 4 ? 2 : 1;
    f.prep = ws.p + at.prep;
    f.rows = ws.p + at.rows;
    f.timeouts = wait_counter();
    auto bits = [&](size_t off) { return reinterpret_cast<unsigned *>(ws.p + off); };
    int st = f.timeouts ? dispatch_prep<Tin>(f, s) : int(SSM_ERR_CUDA);
    f.smax = bits(at.smax); f.emax = bits(at.emax);
    f.v = v; f.e16 = ws.p + at.e16; f.s16 = ws.p + at.s16;
    // segments: whole spans of the kept states
    int nseg = 1;
    if (at.nseg > 1) {
        constexpr int span = ssm::kDeltaSave / ssm::kDeltaC;
        const int chunks = int(delta_chunks(f.seqlen));
        f.seg_chunks = ((chunks + at.nseg - 1) / at.nseg + span - 1) / span * span;
        nseg = (chunks + f.seg_chunks - 1) / f.seg_chunks;
        f.seg_state = part(at.seg_state); f.seg_map = part(at.seg_map);
        if (st == SSM_OK) st = dispatch_chain<KP, Tin, float, 3>(f, s, nseg);
        if (st == SSM_OK) st = launch_fold<false>(f, nseg, s);
    }
    if (st == SSM_OK) st = dispatch_chain<KP, Tin, float, 1>(f, s, nseg);
    if (st == SSM_OK) {
        ssm::DeltaArgs r = f;
        r.v = dy; r.y = dv; r.h0 = dfinal; r.hN = dh0;
        r.d16 = ws.p + at.d16; r.w16 = ws.p + at.w16; r.y16 = ws.p + at.y16;
        r.smax = bits(at.dsmax); r.emax = bits(at.wmax); r.ymax = bits(at.ymax);
        if (nseg > 1) {
            st = dispatch_chain<KP, Tg, float, 4>(r, s, nseg);
            if (st == SSM_OK) st = launch_fold<true>(r, nseg, s);
        }
        if (st == SSM_OK) st = dispatch_chain<KP, Tg, Tg, 2>(r, s, nseg);
    }
    if (st == SSM_OK) {
        const ssm::DeltaGradArgs g{f.a, f.beta, f.rows, f.prep, ws.p + at.e16, ws.p + at.w16, ws.p + at.y16,
                                   ws.p + at.s16, ws.p + at.d16, f.timeouts, bits(at.smax),
                                   bits(at.dsmax), bits(at.emax), bits(at.wmax), bits(at.ymax), part(at.part), dq, dk,
                                   da, dbeta, f.batch, f.seqlen, f.heads, f.qk_heads, f.P, f.N,
                                   delta_slices(f.P) * kDeltaWarps, f.scale};
        st = f.P <= 64 ? dispatch_grad<64, Tin, Tg>(g, s) : dispatch_grad<128, Tin, Tg>(g, s);
    }
    return ws.release(st);
}

}  // namespace

extern "C" {

size_t ssm_delta_rule_bwd_workspace(int batch, int seqlen, int heads, int qk_heads, int headdim, int dstate,
                                    int in_dtype, int grad_dtype) {
    if (!valid_dtype(in_dtype) || !valid_dtype(grad_dtype)) return 0;
    if (delta_sizes(batch, seqlen, heads, qk_heads, headdim, dstate) != SSM_OK) return 0;
    return BwdParts(batch, seqlen, heads, qk_heads, headdim, dstate, in_dtype, grad_dtype).all;
}

int ssm_delta_rule_bwd(const void *q, const void *k, const void *v, const float *a, const float *beta,
                       const float *initial_state, const void *dy, const float *dfinal_state,
                       void *dq, void *dk, void *dv, float *da, float *dbeta, float *dinitial_state,
                       float scale, int batch, int seqlen, int heads, int qk_heads, int headdim, int dstate,
                       int in_dtype, int grad_dtype, void *workspace, size_t workspace_bytes, void *cuda_stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(grad_dtype)) return SSM_ERR_INVALID_ARG;
    if (const int st = delta_sizes(batch, seqlen, heads, qk_heads, headdim, dstate)) return st;
    const long long all = (long long)batch * heads;
    const bool work = all > 0 && seqlen > 0;
    if (work && (!q || !k || !v || !a || !beta || !dy || !dq || !dk || !dv || !da || !dbeta)) return SSM_ERR_INVALID_ARG;
    const size_t tok = size_t(batch) * seqlen, is = dtype_size(in_dtype), gs = dtype_size(grad_dtype);
    const size_t kn = tok * qk_heads * dstate, vn = tok * heads * headdim, hn = tok * heads;
    const size_t sb = size_t(all) * headdim * dstate * 4;
    const struct { const void *p; size_t n; } in[] = {
        {q, kn * is}, {k, kn * is}, {v, vn * is}, {a, hn * 4}, {beta, hn * 4}, {initial_state, sb}, {dy, vn * gs},
        {dfinal_state, sb}};
    const struct { const void *p; size_t n; } out[] = {{dq, kn * gs}, {dk, kn * gs}, {dv, vn * gs}, {da, hn * 4},
                                                       {dbeta, hn * 4}, {dinitial_state, sb}};
    for (const auto &x : in)
        if (x.p && !aligned16(x.p)) return SSM_ERR_ALIGNMENT;
    for (const auto &x : out)
        if (x.p && !aligned16(x.p)) return SSM_ERR_ALIGNMENT;
    if (workspace && !aligned16(workspace)) return SSM_ERR_ALIGNMENT;
    if (all == 0) return SSM_OK;
    for (const auto &x : in)
        if (overlaps(workspace, workspace_bytes, x.p, x.n)) return SSM_ERR_INVALID_ARG;
    for (const auto &x : out)
        if (overlaps(workspace, workspace_bytes, x.p, x.n)) return SSM_ERR_INVALID_ARG;
    for (const auto &x : out) {
        for (const auto &y : in)
            if (overlaps(x.p, x.n, y.p, y.n)) return SSM_ERR_INVALID_ARG;
        for (const auto &y : out)
            if (&x != &y && overlaps(x.p, x.n, y.p, y.n)) return SSM_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    if (!work) {   // no tokens: the start state's gradient is the final state's
        if (!dinitial_state) return SSM_OK;
        if (dfinal_state) return status_of(cudaMemcpyAsync(dinitial_state, dfinal_state, sb, cudaMemcpyDeviceToDevice, s));
        return status_of(cudaMemsetAsync(dinitial_state, 0, sb, s));
    }
    ssm::DeltaArgs f{};
    f.q = q; f.k = k; f.a = a; f.beta = beta; f.h0 = initial_state;
    f.batch = batch; f.seqlen = seqlen; f.heads = heads; f.qk_heads = qk_heads; f.P = headdim; f.N = dstate;
    f.scale = scale;
    using bf16 = __nv_bfloat16;
    if (in_dtype == SSM_BF16)
        return grad_dtype == SSM_BF16 ? run_bwd<bf16, bf16>(f, v, dy, dfinal_state, dq, dk, dv, da, dbeta, dinitial_state, workspace,
                                                                workspace_bytes, s)
                                      : run_bwd<bf16, float>(f, v, dy, dfinal_state, dq, dk, dv, da, dbeta, dinitial_state, workspace,
                                                                workspace_bytes, s);
    return grad_dtype == SSM_BF16 ? run_bwd<float, bf16>(f, v, dy, dfinal_state, dq, dk, dv, da, dbeta, dinitial_state, workspace,
                                                                workspace_bytes, s)
                                  : run_bwd<float, float>(f, v, dy, dfinal_state, dq, dk, dv, da, dbeta, dinitial_state, workspace,
                                                                workspace_bytes, s);
}

}  // extern "C"
