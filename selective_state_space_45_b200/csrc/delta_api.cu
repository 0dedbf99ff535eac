// delta_api.cu -- C ABI of the gated delta rule over whole sequences (ssm_delta_rule_fwd) and
// over decode tokens (ssm_delta_rule_step).  Arguments are checked on the host before
// anything is launched.  The forward takes scratch (the caller's workspace or a stream-ordered
// buffer), the step none.
#include <algorithm>

#include "delta_host.cuh"
#include "delta_step.cuh"

using namespace ssm_host;

namespace {

template <typename Tin, typename Tout> int launch_step(const ssm::DeltaStepArgs &a, cudaStream_t s) {
    const long long blocks = ((long long)a.batch * a.heads * (a.P / 8) + 7) / 8;
    if (blocks > INT_MAX) return SSM_ERR_UNSUPPORTED;
    const unsigned n = unsigned(blocks);
    if (a.N <= 32) ssm::delta_step_kernel<1, Tin, Tout><<<n, 256, 0, s>>>(a);
    else if (a.N <= 64) ssm::delta_step_kernel<2, Tin, Tout><<<n, 256, 0, s>>>(a);
    else if (a.N <= 96) ssm::delta_step_kernel<3, Tin, Tout><<<n, 256, 0, s>>>(a);
    else ssm::delta_step_kernel<4, Tin, Tout><<<n, 256, 0, s>>>(a);
    return status_of(cudaGetLastError());
}

struct FwdPlan {
    int nseg;
    size_t prep, rows, seg_state, seg_map, all;      // offsets, and the bytes
    FwdPlan(int batch, int seqlen, int heads, int qk_heads, int P, int N, int in_dtype) {
        nseg = segments(batch, seqlen, heads, P, N, in_dtype == SSM_F32, false);
        const size_t seg = nseg > 1 ? size_t(batch) * heads * nseg * N * 4 : 0;
        prep = 0;
        rows = prep + round16(prep_bytes(batch, seqlen, heads));
        seg_state = rows + round16(rows_bytes(batch, seqlen, qk_heads, N, in_dtype));
        seg_map = seg_state + seg * P;
        all = seg_map + seg * N;
    }
};

// Forward: the chunk blocks and operands, then the chains, in segments where that pays.
template <typename Tin, typename Tout> int run_fwd(ssm::DeltaArgs a, void *workspace, size_t bytes, cudaStream_t s) {
    const FwdPlan at(a.batch, a.seqlen, a.heads, a.qk_heads, a.P, a.N, sizeof(Tin) == 4 ? SSM_F32 : SSM_BF16);
    constexpr int KP = sizeof(Tin) == 4 ? 2 : 1;
    Scratch ws;
    if (const int st = ws.take(workspace, bytes, at.all, s)) return st;
    a.prep = ws.p + at.prep;
    a.rows = ws.p + at.rows;
    a.seg_state = reinterpret_cast<float *>(ws.p + at.seg_state);
    a.seg_map = reinterpret_cast<float *>(ws.p + at.seg_map);
    a.timeouts = wait_counter();
    int st = a.timeouts ? dispatch_prep<Tin>(a, s) : int(SSM_ERR_CUDA);
    if (at.nseg > 1) {
        const long long chunks = (long long)delta_chunks(a.seqlen);
        a.seg_chunks = int((chunks + at.nseg - 1) / at.nseg);
        const int nseg = int((chunks + a.seg_chunks - 1) / a.seg_chunks);
        if (st == SSM_OK) st = dispatch_chain<KP, Tin, Tout, 3>(a, s, nseg);
        if (st == SSM_OK) st = launch_fold<false>(a, nseg, s);
        // a state carried in place: the last segment's end must not be written before the first
        // segment has read its start, so it goes by the slot that the last segment leaves unused
        float *const end = a.hN;
        const size_t state = size_t(a.P) * a.N * 4;
        const bool in_place = end != nullptr && end == a.h0;
        a.end_slot = in_place;
        if (st == SSM_OK) st = dispatch_chain<KP, Tin, Tout, 0>(a, s, nseg);
        if (st == SSM_OK && in_place)
            st = status_of(cudaMemcpy2DAsync(end, state, ws.p + at.seg_state + (nseg - 1) * state, nseg * state, state,
                                             size_t(a.batch) * a.heads, cudaMemcpyDeviceToDevice, s));
    } else if (st == SSM_OK) {
        st = dispatch_chain<KP, Tin, Tout, 0>(a, s);
    }
    return ws.release(st);
}

}  // namespace

extern "C" {

size_t ssm_delta_rule_fwd_workspace(int batch, int seqlen, int heads, int qk_heads, int headdim, int dstate,
                                    int in_dtype, int out_dtype) {
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return 0;
    if (delta_sizes(batch, seqlen, heads, qk_heads, headdim, dstate) != SSM_OK) return 0;
    if (batch == 0 || heads == 0 || seqlen == 0) return 0;
    return FwdPlan(batch, seqlen, heads, qk_heads, headdim, dstate, in_dtype).all;
}

int ssm_delta_rule_fwd(const void *q, const void *k, const void *v, const float *a, const float *beta,
                       void *y, const float *initial_state, float *final_state, float scale,
                       int batch, int seqlen, int heads, int qk_heads, int headdim, int dstate,
                       int in_dtype, int out_dtype, void *workspace, size_t workspace_bytes, void *cuda_stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return SSM_ERR_INVALID_ARG;
    if (const int st = delta_sizes(batch, seqlen, heads, qk_heads, headdim, dstate)) return st;
    const long long all = (long long)batch * heads;
    const bool work = all > 0 && seqlen > 0;
    if (work && (!q || !k || !v || !a || !beta || !y)) return SSM_ERR_INVALID_ARG;
    for (const void *x : {q, k, v, (const void *)a, (const void *)beta, (const void *)y, (const void *)initial_state,
                          (const void *)final_state, (const void *)workspace})
        if (x && !aligned16(x)) return SSM_ERR_ALIGNMENT;
    if (all == 0) return SSM_OK;
    const size_t tok = size_t(batch) * seqlen, is = dtype_size(in_dtype), os = dtype_size(out_dtype);
    const size_t sb = size_t(all) * headdim * dstate * 4, yb = tok * heads * headdim * os;
    const struct { const void *p; size_t n; } in[] = {
        {q, tok * qk_heads * dstate * is}, {k, tok * qk_heads * dstate * is}, {v, tok * heads * headdim * is},
        {a, tok * heads * 4}, {beta, tok * heads * 4}};
    for (const auto &x : in)
        if (overlaps(y, yb, x.p, x.n) || overlaps(final_state, sb, x.p, x.n)) return SSM_ERR_INVALID_ARG;
    for (const auto &x : in)
        if (overlaps(workspace, workspace_bytes, x.p, x.n)) return SSM_ERR_INVALID_ARG;
    if (overlaps(workspace, workspace_bytes, y, yb) || overlaps(workspace, workspace_bytes, final_state, sb) ||
        overlaps(workspace, workspace_bytes, initial_state, sb))
        return SSM_ERR_INVALID_ARG;
    if (overlaps(y, yb, initial_state, sb) || overlaps(y, yb, final_state, sb)) return SSM_ERR_INVALID_ARG;
    if (final_state != initial_state && overlaps(final_state, sb, initial_state, sb)) return SSM_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    if (!work) {   // no tokens: the final state is the start state
        if (!final_state || final_state == initial_state) return SSM_OK;
        if (initial_state) return status_of(cudaMemcpyAsync(final_state, initial_state, sb, cudaMemcpyDeviceToDevice, s));
        return status_of(cudaMemsetAsync(final_state, 0, sb, s));
    }
    ssm::DeltaArgs g{};
    g.q = q; g.k = k; g.v = v; g.a = a; g.beta = beta; g.y = y; g.h0 = initial_state; g.hN = final_state;
    g.batch = batch; g.seqlen = seqlen; g.heads = heads; g.qk_heads = qk_heads; g.P = headdim; g.N = dstate;
    g.scale = scale;
    using bf16 = __nv_bfloat16;
    if (in_dtype == SSM_BF16)
        return out_dtype == SSM_BF16 ? run_fwd<bf16, bf16>(g, workspace, workspace_bytes, s)
                                     : run_fwd<bf16, float>(g, workspace, workspace_bytes, s);
    return out_dtype == SSM_BF16 ? run_fwd<float, bf16>(g, workspace, workspace_bytes, s)
                                 : run_fwd<float, float>(g, workspace, workspace_bytes, s);
}

int ssm_delta_rule_step(float *state, const void *q, const void *k, const void *v, const float *a,
                        const float *beta, void *y, float scale, int ntok, int batch, int heads,
                        int qk_heads, int headdim, int dstate, int in_dtype, int out_dtype,
                        void *cuda_stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return SSM_ERR_INVALID_ARG;
    if (const int st = delta_sizes(batch, ntok, heads, qk_heads, headdim, dstate)) return st;
    const long long all = (long long)batch * heads;
    if (all == 0 || ntok == 0) return SSM_OK;
    if (!state || !q || !k || !v || !a || !beta || !y) return SSM_ERR_INVALID_ARG;
    for (const void *x : {(const void *)state, q, k, v, (const void *)a, (const void *)beta, (const void *)y})
        if (!aligned16(x)) return SSM_ERR_ALIGNMENT;
    const size_t tok = size_t(batch) * ntok, is = dtype_size(in_dtype);
    const size_t sb = size_t(all) * headdim * dstate * 4, yb = tok * heads * headdim * dtype_size(out_dtype);
    const struct { const void *p; size_t n; } in[] = {
        {q, tok * qk_heads * dstate * is}, {k, tok * qk_heads * dstate * is}, {v, tok * heads * headdim * is},
        {a, tok * heads * 4}, {beta, tok * heads * 4}};
    for (const auto &x : in)
        if (overlaps(y, yb, x.p, x.n) || overlaps(state, sb, x.p, x.n)) return SSM_ERR_INVALID_ARG;
    if (overlaps(y, yb, state, sb)) return SSM_ERR_INVALID_ARG;
    const ssm::DeltaStepArgs g{state, q, k, v, a, beta, y, ntok, batch, heads, qk_heads, headdim, dstate, scale};
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    using bf16 = __nv_bfloat16;
    if (in_dtype == SSM_BF16) return out_dtype == SSM_BF16 ? launch_step<bf16, bf16>(g, s) : launch_step<bf16, float>(g, s);
    return out_dtype == SSM_BF16 ? launch_step<float, bf16>(g, s) : launch_step<float, float>(g, s);
}

}  // extern "C"
