// delta_bwd_api.cu -- C ABI of the gated delta rule's backward (ssm_delta_rule_bwd): the
// forward pass again (e and the states every 64 tokens), the reverse pass (dv, the state's
// gradient at the same places), then the chunks' gradients in parallel.  One stream-ordered
// scratch buffer per call.
#include "delta_grad.cuh"
#include "delta_host.cuh"

using namespace ssm_host;

namespace {

template <int NP, typename Tin, typename Tg> int launch_grad(const ssm::DeltaGradArgs &a, cudaStream_t s) {
    const long long ctas = (long long)a.batch * a.qk_heads * ((a.seqlen + ssm::kGradC - 1) / ssm::kGradC);
    if (ctas > INT_MAX) return SSM_ERR_UNSUPPORTED;
    constexpr int smem = ssm::delta_grad_smem<NP>();
    if (cudaFuncSetAttribute(ssm::delta_grad_kernel<NP, Tin, Tg>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return SSM_ERR_CUDA;
    ssm::delta_grad_kernel<NP, Tin, Tg><<<unsigned(ctas), 256, smem, s>>>(a);
    return status_of(cudaGetLastError());
}

template <typename Tin, typename Tg>
int run_bwd(ssm::DeltaArgs f, const void *v, const void *dy, const float *dfinal, void *dq, void *dk, void *dv, float *da,
            float *dbeta, float *dh0, cudaStream_t s) {
    const size_t all = size_t(f.batch) * f.heads, tok = all * f.seqlen;
    const size_t nbound = (size_t(f.seqlen) + ssm::kDeltaSave - 1) / ssm::kDeltaSave + 1;
    const int slices = (f.P + 63) / 64, zparts = 4 * slices;
    const size_t n_e = tok * f.P, n_w = sizeof(Tg) == 4 ? 0 : n_e, n_ck = all * nbound * f.P * f.N;
    const size_t n_sum = size_t(slices) * tok, n_z = size_t(zparts) * all * nbound;
    auto up = [](size_t n) { return (n + 3) / 4 * 4; };        // 16-byte parts
    float *ws = nullptr;
    if (cudaMallocAsync(reinterpret_cast<void **>(&ws),
                        (up(n_e) + up(n_w) + 2 * up(n_ck) + 3 * up(n_sum) + up(n_z)) * sizeof(float), s) != cudaSuccess) {
        cudaGetLastError();
        return SSM_ERR_CUDA;
    }
    float *at = ws;
    auto take = [&](size_t n) { float *r = at; at += up(n); return r; };
    float *e = take(n_e), *w = n_w ? take(n_w) : static_cast<float *>(dv), *ck = take(n_ck), *dck = take(n_ck);
    float *dyy = take(n_sum), *vw = take(n_sum), *edu = take(n_sum), *zsum = take(n_z);

    f.v = v; f.v2 = dy; f.y = nullptr; f.hN = nullptr; f.e = e; f.ck = ck; f.sum0 = dyy;
    int st = dispatch_chain<Tin, Tin, Tg, float, 1>(f, s);
    if (st == SSM_OK) {
        ssm::DeltaArgs r = f;
        r.v = dy; r.v2 = v; r.y = dv; r.h0 = dfinal; r.hN = dh0; r.w = n_w ? w : nullptr; r.dck = dck;
        r.sum0 = vw; r.sum1 = edu; r.zsum = zsum;
        st = dispatch_chain<Tin, Tg, Tin, Tg, 2>(r, s);
    }
    if (st == SSM_OK) {
        const ssm::DeltaGradArgs g{f.q, f.k, dy, f.a, f.beta, e, w, ck, dck, dyy, vw, edu, zsum, dq, dk, da, dbeta,
                                   f.batch, f.seqlen, f.heads, f.qk_heads, f.P, f.N, slices, zparts, f.scale};
        st = f.N <= 64 ? launch_grad<64, Tin, Tg>(g, s) : launch_grad<128, Tin, Tg>(g, s);
    }
    const cudaError_t fe = cudaFreeAsync(ws, s);
    return st == SSM_OK && fe != cudaSuccess ? int(SSM_ERR_CUDA) : st;
}

}  // namespace

extern "C" {

int ssm_delta_rule_bwd(const void *q, const void *k, const void *v, const float *a, const float *beta,
                       const float *initial_state, const void *dy, const float *dfinal_state,
                       void *dq, void *dk, void *dv, float *da, float *dbeta, float *dinitial_state,
                       float scale, int batch, int seqlen, int heads, int qk_heads, int headdim, int dstate,
                       int in_dtype, int grad_dtype, void *cuda_stream) {
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
    if (all == 0) return SSM_OK;
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
        return grad_dtype == SSM_BF16 ? run_bwd<bf16, bf16>(f, v, dy, dfinal_state, dq, dk, dv, da, dbeta, dinitial_state, s)
                                      : run_bwd<bf16, float>(f, v, dy, dfinal_state, dq, dk, dv, da, dbeta, dinitial_state, s);
    return grad_dtype == SSM_BF16 ? run_bwd<float, bf16>(f, v, dy, dfinal_state, dq, dk, dv, da, dbeta, dinitial_state, s)
                                  : run_bwd<float, float>(f, v, dy, dfinal_state, dq, dk, dv, da, dbeta, dinitial_state, s);
}

}  // extern "C"
