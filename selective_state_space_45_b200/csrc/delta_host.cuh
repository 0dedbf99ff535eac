// delta_host.cuh -- what the delta rule's entry points share on the host.
#pragma once

#include <climits>

#include "api_host.cuh"
#include "delta_rule.cuh"

namespace ssm_host {

// Sizes of a call; `tokens` is seqlen, or the tokens of a step.
inline int delta_sizes(int batch, int tokens, int heads, int qk_heads, int headdim, int dstate) {
    if (batch < 0 || tokens < 0 || heads < 0 || qk_heads < 0 || headdim < 1 || dstate < 1) return SSM_ERR_INVALID_ARG;
    if (heads > 0 && (qk_heads == 0 || heads % qk_heads != 0)) return SSM_ERR_INVALID_ARG;
    if (headdim % 8 != 0 || dstate % 8 != 0 || headdim > 256 || dstate > 128) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

// The chain kernel for one set of types: a warp per 16 rows of the state, four of them and
// the producer per CTA.
template <int NP, typename Tin, typename Tv, typename Tv2, typename Tout, int MODE>
int launch_chain(ssm::DeltaArgs a, cudaStream_t s) {
    using Cfg = ssm::DeltaCfg<NP, 4, Tin, Tv, Tv2, Tout, MODE>;
    a.slices = (a.P + 16 * Cfg::NW - 1) / (16 * Cfg::NW);
    const long long ctas = (long long)a.batch * a.heads * a.slices;
    if (ctas > INT_MAX) return SSM_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(ssm::delta_chain_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(Cfg::SMEM_BYTES)) != cudaSuccess)
        return SSM_ERR_CUDA;
    ssm::delta_chain_kernel<Cfg><<<unsigned(ctas), Cfg::NT, Cfg::SMEM_BYTES, s>>>(a);
    return status_of(cudaGetLastError());
}

// dstate padded to the next multiple of 32 (zero columns): the products' inner length.
template <typename Tin, typename Tv, typename Tv2, typename Tout, int MODE>
int dispatch_chain(const ssm::DeltaArgs &a, cudaStream_t s) {
    if (a.N <= 32) return launch_chain<32, Tin, Tv, Tv2, Tout, MODE>(a, s);
    if (a.N <= 64) return launch_chain<64, Tin, Tv, Tv2, Tout, MODE>(a, s);
    if (a.N <= 96) return launch_chain<96, Tin, Tv, Tv2, Tout, MODE>(a, s);
    return launch_chain<128, Tin, Tv, Tv2, Tout, MODE>(a, s);
}

}  // namespace ssm_host
