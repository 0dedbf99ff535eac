// norm_api.cu -- C ABI of the layer norm (ssm_layer_norm_fwd, ssm_layer_norm_bwd).
#include <algorithm>
#include <type_traits>

#include "api_scratch.cuh"
#include "layer_norm.cuh"

using namespace ssm_host;

namespace {

constexpr int kSMs = 148, kMaxDim = 8192;

// The group that owns a row and its vectors per lane, by the row's width: f(lanes, V, threads)
// with `lanes` 8 or 32 within a warp (CTAs of 256 threads), or 0 for one CTA per row.  A
// backward lane carries 16 V column sums beside the row, so its warps stop at V = 2.  A warp per
// row where it can be: 16384 rows of 768 take 16.4 us with the call and 22.5 with a CTA per row.
template <bool BWD, typename F> int by_width(int dim, F f) {
    using std::integral_constant;
    if (dim <= 64) return f(integral_constant<int, 8>(), integral_constant<int, 1>(), 256);
    if (dim <= 128) return f(integral_constant<int, 8>(), integral_constant<int, 2>(), 256);
    if (dim <= 256) return f(integral_constant<int, 32>(), integral_constant<int, 1>(), 256);
    if (dim <= 512) return f(integral_constant<int, 32>(), integral_constant<int, 2>(), 256);
    if constexpr (!BWD) {
        if (dim <= 768) return f(integral_constant<int, 32>(), integral_constant<int, 3>(), 256);
        if (dim <= 1024) return f(integral_constant<int, 32>(), integral_constant<int, 4>(), 256);
    }
    return f(integral_constant<int, 0>(), integral_constant<int, 2>(), (dim + 511) / 512 * 32);
}

// CTAs: one for the rows it takes, at most what the GPU's SMs hold at `per_sm` threads each (a CTA
// walks the rest of its rows).
int grid_of(int lanes, int threads, int per_sm, int rows) {
    const int per_cta = lanes ? threads / lanes : 1;
    return std::min((rows - 1) / per_cta + 1, kSMs * std::max(1, per_sm / threads));
}

// Threads of a kernel that an SM's registers hold at once.
template <typename K> int resident(K kernel) {
    cudaFuncAttributes at{};
    if (cudaFuncGetAttributes(&at, kernel) != cudaSuccess) { cudaGetLastError(); return 512; }
    return std::min(2048, 65536 / ((std::max(at.numRegs, 32) + 7) / 8 * 8) / 32 * 32);
}

// Narrow rows go several a step once the whole grid has that many for every group: 393216 rows
// of 64 took 26.6 us so and 28.7 one by one, 98304 rows of 256 26.7 and 28.7 (bf16, from HBM); with
// fewer the idle places cost more than they bring (1000 rows of 64: 8.2 and 6.1 us), and so they
// do where a lane's values are loaded one by one (393219 rows of 63: 47 and 43 us).
template <bool VEC, typename Tin, typename Tout> int run_fwd(const ssm::NormArgs &a, cudaStream_t s) {
    return by_width<false>(a.dim, [&](auto lanes, auto v, int threads) {
        constexpr int R = !VEC ? 1 : lanes() == 8 && v() == 1 ? 4 : lanes() == 8 || (lanes() == 32 && v() == 1) ? 2 : 1;
        if constexpr (R > 1) {
            auto kernel = ssm::layer_norm_fwd_kernel<lanes(), v(), R, VEC, Tin, Tout>;
            static const int per_sm = resident(kernel);
            const int grid = kSMs * std::max(1, per_sm / threads);
            if (a.rows >= (long long)grid * (threads / lanes()) * R) {
                kernel<<<grid, threads, 0, s>>>(a);
                return status_of(cudaGetLastError());
            }
        }
        auto kernel = ssm::layer_norm_fwd_kernel<lanes(), v(), 1, VEC, Tin, Tout>;
        static const int per_sm = resident(kernel);
        kernel<<<grid_of(lanes(), threads, per_sm, int(a.rows)), threads, 0, s>>>(a);
        return status_of(cudaGetLastError());
    });
}

// The backward's CTAs at most, whatever the types: what the workspace has room for.
constexpr int kBwdPerSm = 512;
int bwd_grid(int rows, int dim) {
    return by_width<true>(dim, [&](auto lanes, auto, int threads) { return grid_of(lanes(), threads, kBwdPerSm, rows); });
}

template <bool VEC, typename Tin, typename Tg>
int run_bwd(ssm::NormArgs a, float *dw, float *db, void *workspace, size_t bytes, cudaStream_t s) {
    int grid = 0;
    Scratch ws;
    if (const int st = ws.take(workspace, bytes, ssm_layer_norm_bwd_workspace(int(a.rows), a.dim), s)) return st;
    a.part = reinterpret_cast<float *>(ws.p);
    int st = by_width<true>(a.dim, [&](auto lanes, auto v, int threads) {
        auto kernel = ssm::layer_norm_bwd_kernel<lanes(), v(), VEC, Tin, Tg>;
        // one wave: rows of 257 to 512 values with an fp32 side take 150 registers a thread, which one
        // CTA of 256 fits and two do not (65536 rows of 512, fp32: 92.0 us in two waves, 83.2 so)
        static const int per_sm = std::min(kBwdPerSm, resident(kernel));
        grid = grid_of(lanes(), threads, per_sm, int(a.rows));
        kernel<<<grid, threads, lanes() ? 2 * size_t(a.dim) * sizeof(float) : 0, s>>>(a);
        return status_of(cudaGetLastError());
    });
    if (st == SSM_OK && (dw != nullptr || db != nullptr)) {
        ssm::layer_norm_cols_kernel<<<(2 * a.dim + 31) / 32, 1024, 0, s>>>(a.part, grid, a.dim, dw, db);
        st = status_of(cudaGetLastError());
    }
    return ws.release(st);
}

template <typename F> int by_types(int ta, int tb, F f) {
    using bf16 = __nv_bfloat16;
    if (ta == SSM_F32) return tb == SSM_F32 ? f(float(), float()) : f(float(), bf16());
    return tb == SSM_F32 ? f(bf16(), float()) : f(bf16(), bf16());
}

}  // namespace

extern "C" {

int ssm_layer_norm_fwd(const void *x, const float *weight, const float *bias, void *y, float *mean,
                       float *rstd, float eps, int rows, int dim, int in_dtype, int out_dtype,
                       void *cuda_stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return SSM_ERR_INVALID_ARG;
    if (rows < 0 || dim < 1 || !(eps >= 0.f)) return SSM_ERR_INVALID_ARG;
    if (dim > kMaxDim) return SSM_ERR_UNSUPPORTED;
    if (rows > 0 && (!x || !y)) return SSM_ERR_INVALID_ARG;
    for (const void *q : {x, (const void *)weight, (const void *)bias, (const void *)y, (const void *)mean, (const void *)rstd})
        if (q && !aligned16(q)) return SSM_ERR_ALIGNMENT;
    const size_t n = size_t(rows) * dim, wb = size_t(dim) * 4, sb = size_t(rows) * 4;
    const struct { const void *p; size_t n; } in[] = {{x, n * dtype_size(in_dtype)}, {weight, wb}, {bias, wb}};
    const struct { const void *p; size_t n; } out[] = {{y, n * dtype_size(out_dtype)}, {mean, sb}, {rstd, sb}};
    for (const auto &o : out) {
        for (const auto &q : in)
            if (overlaps(o.p, o.n, q.p, q.n)) return SSM_ERR_INVALID_ARG;
        for (const auto &q : out)
            if (&o != &q && overlaps(o.p, o.n, q.p, q.n)) return SSM_ERR_INVALID_ARG;
    }
    if (rows == 0) return SSM_OK;
    ssm::NormArgs a{};
    a.x = x; a.w = weight; a.b = bias; a.out = y; a.mean = mean; a.rstd = rstd; a.rows = rows; a.dim = dim; a.eps = eps;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return by_types(in_dtype, out_dtype, [&](auto ti, auto to) {
        using Ti = decltype(ti);
        using To = decltype(to);
        return dim % 8 == 0 ? run_fwd<true, Ti, To>(a, s) : run_fwd<false, Ti, To>(a, s);
    });
}

size_t ssm_layer_norm_bwd_workspace(int rows, int dim) {
    if (rows < 1 || dim < 1 || dim > kMaxDim) return 0;
    return size_t(bwd_grid(rows, dim)) * 2 * dim * sizeof(float);
}

int ssm_layer_norm_bwd(const void *dy, const void *x, const float *weight, const float *mean,
                       const float *rstd, void *dx, float *dweight, float *dbias, int rows, int dim,
                       int in_dtype, int grad_dtype, void *workspace, size_t workspace_bytes, void *cuda_stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(grad_dtype)) return SSM_ERR_INVALID_ARG;
    if (rows < 0 || dim < 1) return SSM_ERR_INVALID_ARG;
    if (dim > kMaxDim) return SSM_ERR_UNSUPPORTED;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return SSM_ERR_INVALID_ARG;
    for (const void *q : {dy, x, (const void *)weight, (const void *)mean, (const void *)rstd, (const void *)dx,
                          (const void *)dweight, (const void *)dbias, (const void *)workspace})
        if (q && !aligned16(q)) return SSM_ERR_ALIGNMENT;
    const size_t n = size_t(rows) * dim, wb = size_t(dim) * 4, sb = size_t(rows) * 4, gb = n * dtype_size(grad_dtype);
    const struct { const void *p; size_t n; } in[] = {{x, n * dtype_size(in_dtype)}, {weight, wb}, {dy, gb}, {mean, sb}, {rstd, sb}};
    const struct { const void *p; size_t n; } out[] = {{dx, gb}, {dweight, wb}, {dbias, wb}};
    for (const auto &q : in)
        if (overlaps(workspace, workspace_bytes, q.p, q.n)) return SSM_ERR_INVALID_ARG;
    for (const auto &o : out) {
        if (overlaps(workspace, workspace_bytes, o.p, o.n)) return SSM_ERR_INVALID_ARG;
        for (const auto &q : in)
            if (overlaps(o.p, o.n, q.p, q.n)) return SSM_ERR_INVALID_ARG;
        for (const auto &q : out)
            if (&o != &q && overlaps(o.p, o.n, q.p, q.n)) return SSM_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    if (rows == 0) {   // no rows: the sums over them are zero
        if (dweight && cudaMemsetAsync(dweight, 0, wb, s) != cudaSuccess) return SSM_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, wb, s) != cudaSuccess) return SSM_ERR_CUDA;
        return SSM_OK;
    }
    ssm::NormArgs a{};
    a.x = x; a.dy = dy; a.w = weight; a.out = dx; a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.rows = rows; a.dim = dim;
    return by_types(in_dtype, grad_dtype, [&](auto ti, auto tg) {
        using Ti = decltype(ti);
        using Tg = decltype(tg);
        return dim % 8 == 0 ? run_bwd<true, Ti, Tg>(a, dweight, dbias, workspace, workspace_bytes, s)
                            : run_bwd<false, Ti, Tg>(a, dweight, dbias, workspace, workspace_bytes, s);
    });
}

}  // extern "C"
