// delta_host.cuh -- what the delta rule's entry points share on the host.
#pragma once

#include <climits>
#include <cmath>

#include "api_scratch.cuh"
#include "delta_rule.cuh"

namespace ssm_host {

// Sizes of a call; `tokens` is seqlen, or the tokens of a step.
inline int delta_sizes(int batch, int tokens, int heads, int qk_heads, int headdim, int dstate) {
    if (batch < 0 || tokens < 0 || heads < 0 || qk_heads < 0 || headdim < 1 || dstate < 1) return SSM_ERR_INVALID_ARG;
    if (heads > 0 && (qk_heads == 0 || heads % qk_heads != 0)) return SSM_ERR_INVALID_ARG;
    if (tokens > INT_MAX - 128) return SSM_ERR_UNSUPPORTED;
    if (headdim % 8 != 0 || dstate % 8 != 0 || headdim > 128 || dstate > 128) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

inline size_t delta_chunks(int seqlen) { return (size_t(seqlen) + ssm::kDeltaC - 1) / ssm::kDeltaC; }

// Bytes of the prep kernel's blocks.
inline size_t prep_bytes(int batch, int seqlen, int heads) {
    return size_t(batch) * heads * delta_chunks(seqlen) * ssm::DeltaBlock::BYTES;
}
// dstate padded to the next multiple of 32 (zero columns): the products' inner length.
inline int padded_state(int N) { return (N + 31) / 32 * 32; }

// Bytes of k and q as operands: 32 rows per chunk, two pieces of fp32 ones.
inline size_t rows_bytes(int batch, int seqlen, int qk_heads, int N, int in_dtype) {
    return size_t(batch) * qk_heads * delta_chunks(seqlen) *
           (2 * (in_dtype == SSM_F32 ? 2 : 1) * ssm::kDeltaC * (padded_state(N) * 2 + 16));
}

// Dynamic shared memory of a kernel, with the SM's memory split for as many CTAs as fit (the
// default split left one chain CTA per SM where two fit).
template <typename K> int set_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess &&
                   cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                        int(cudaSharedmemCarveoutMaxShared)) == cudaSuccess
               ? SSM_OK
               : SSM_ERR_CUDA;
}

// The chunk blocks into a.prep, k and q as operands into a.rows.
template <int NP, typename Tin> int launch_prep(const ssm::DeltaArgs &a, cudaStream_t s) {
    const long long blocks = ((long long)a.batch * a.heads * (long long)delta_chunks(a.seqlen) + 3) / 4;
    if (blocks > INT_MAX) return SSM_ERR_UNSUPPORTED;
    constexpr int smem = 4 * int(sizeof(ssm::PrepScratch<NP, Tin>));
    if (const int st = set_smem(ssm::delta_prep_kernel<NP, Tin>, smem)) return st;
    ssm::delta_prep_kernel<NP, Tin><<<unsigned(blocks), 128, smem, s>>>(a);
    return status_of(cudaGetLastError());
}
template <typename Tin> int dispatch_prep(const ssm::DeltaArgs &a, cudaStream_t s) {
    switch (padded_state(a.N)) {
    case 32: return launch_prep<32, Tin>(a, s);
    case 64: return launch_prep<64, Tin>(a, s);
    case 96: return launch_prep<96, Tin>(a, s);
    default: return launch_prep<128, Tin>(a, s);
    }
}

// The chain kernel for one set of types: a warp per 16 rows of the state, four per CTA.
constexpr int kDeltaWarps = 4;
inline int delta_slices(int P) { return (P + 16 * kDeltaWarps - 1) / (16 * kDeltaWarps); }

template <int NP, int KP, typename Tv, typename Tout, int MODE>
int launch_chain(ssm::DeltaArgs a, int nseg, cudaStream_t s) {
    using Cfg = ssm::DeltaCfg<NP, kDeltaWarps, KP, Tv, Tout, MODE>;
    a.slices = delta_slices(a.P);
    if (nseg == 1) a.seg_chunks = int(delta_chunks(a.seqlen));
    // MODE 3 has the identity's rows beside those of headdim
    const long long ctas = (long long)a.batch * a.heads * (a.slices + (MODE == 3 ? delta_slices(a.N) : 0));
    if (ctas > INT_MAX) return SSM_ERR_UNSUPPORTED;
    if (const int st = set_smem(ssm::delta_chain_kernel<Cfg>, int(Cfg::SMEM_BYTES))) return st;
    ssm::delta_chain_kernel<Cfg><<<dim3(unsigned(ctas), unsigned(nseg)), Cfg::NT, Cfg::SMEM_BYTES, s>>>(a);
    return status_of(cudaGetLastError());
}

template <int KP, typename Tv, typename Tout, int MODE>
int dispatch_chain(const ssm::DeltaArgs &a, cudaStream_t s, int nseg = 1) {
    switch (padded_state(a.N)) {
    case 32: return launch_chain<32, KP, Tv, Tout, MODE>(a, nseg, s);
    case 64: return launch_chain<64, KP, Tv, Tout, MODE>(a, nseg, s);
    case 96: return launch_chain<96, KP, Tv, Tout, MODE>(a, nseg, s);
    default: return launch_chain<128, KP, Tv, Tout, MODE>(a, nseg, s);
    }
}

// How many segments a sequence is cut into.  A chain's chunks follow one another, so with few
// heads most of the GPU is idle.  Segments run at once: first every segment's end state from a
// zero start and its map (dstate more rows), then, from the folded start states, the outputs.
// In units of a chunk's time in a CTA (2.0 us; 0.8 of it for end states and maps): two CTAs on an
// SM take 1.8, more share it; fp32 inputs leave room for one CTA.  Folding costs about four units
// a segment.  Segments have at least 16 chunks, and what they save must be a tenth.  32749 tokens
// of 16 heads of 128 x 128: one piece 2090 us, nine segments 1088; 8 heads 2046 and 633; 8192
// tokens of 8 heads in fp32, 726 and 357.  The backward's two passes take 2.5 units a chunk
// together, and its segments need their gradients of the start states (1.1) and a second fold too:
// 8192 tokens of 8 heads of 128 x 128, 1455 us in one piece, 689 in segments; 2 x 4096 of 12 heads
// of 64 x 128, 835 and 599.
inline int segments(int batch, int seqlen, int heads, int P, int N, bool one_per_sm, bool backward) {
    const long long chunks = (long long)delta_chunks(seqlen), all = (long long)batch * heads;
    auto cost = [&](double ctas) {
        const double r = ctas / 148;
        return r <= 1 ? 1.0 : one_per_sm ? std::ceil(r) : r <= 2 ? 1.8 : 0.9 * r;
    };
    const double rows = double(all) * delta_slices(P), maps = double(all) * delta_slices(N);
    const double last = backward ? 2.5 : 1.0;
    int best = 1;
    double least = chunks * last * cost(rows);
    const double bar = 0.9 * least;
    for (int n = 2; n <= 64 && chunks / n >= 16; ++n) {
        const double t = double((chunks + n - 1) / n) * (0.8 * cost((n - 1) * rows + (n - 2) * maps) +
                                                         (backward ? 1.1 * cost((n - 1) * rows) : 0.0) + last * cost(n * rows)) +
                         (backward ? 8 : 4) * n;
        if (t < bar && t < least) { least = t; best = n; }
    }
    return best;
}

// The segments' start states (REV: the gradients of their end states) from what they ended with.
template <bool REV> int launch_fold(const ssm::DeltaArgs &a, int nseg, cudaStream_t s) {
    const unsigned ctas = unsigned(a.batch) * unsigned(a.heads) * unsigned((a.P + 7) / 8);
    ssm::delta_fold_kernel<8, REV><<<ctas, 128, 0, s>>>(a, nseg);
    return status_of(cudaGetLastError());
}

}  // namespace ssm_host
