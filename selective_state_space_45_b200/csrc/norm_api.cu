// norm_api.cu -- C ABI of the layer norm (ssm_layer_norm_fwd, ssm_layer_norm_bwd).
#include <algorithm>
#include <type_traits>

#include "api_host.cuh"
#include "layer_norm.cuh"

using namespace ssm_host;

namespace {

constexpr int kSMs = 148, kMaxDim = 8192;

// The group that owns a row and its vectors per lane, by the row's width: f(lanes, V, threads)
// with `lanes` 8 or 32 within a warp (CTAs of 256 threads), or 0 for one CTA per row.  A
// backward lane carries 16 V column sums beside the row, so its warps stop at V = 2.
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

// CTAs that the GPU holds at once, or fewer if the rows need fewer.
template <typename K> int grid_of(K kernel, int threads, size_t smem, long long rows, int rows_per_cta, int *grid) {
    int per = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess || per < 1)
        return SSM_ERR_CUDA;
    *grid = int(std::min<long long>((rows + rows_per_cta - 1) / rows_per_cta, (long long)kSMs * per));
    return SSM_OK;
}

template <bool VEC, typename Tin, typename Tout> int run_fwd(const ssm::NormArgs &a, cudaStream_t s) {
    return by_width<false>(a.dim, [&](auto lanes, auto v, int threads) {
        auto kernel = ssm::layer_norm_fwd_kernel<lanes(), v(), VEC, Tin, Tout>;
        int grid = 0;
        if (const int st = grid_of(kernel, threads, 0, a.rows, lanes() ? threads / std::max(1, lanes()) : 1, &grid)) return st;
        kernel<<<grid, threads, 0, s>>>(a);
        return status_of(cudaGetLastError());
    });
}

template <bool VEC, typename Tin, typename Tg>
int run_bwd(ssm::NormArgs a, float *dw, float *db, cudaStream_t s) {
    return by_width<true>(a.dim, [&](auto lanes, auto v, int threads) {
        auto kernel = ssm::layer_norm_bwd_kernel<lanes(), v(), VEC, Tin, Tg>;
        const size_t smem = lanes() ? 2 * size_t(a.dim) * sizeof(float) : 0;
        int grid = 0;
        if (const int st = grid_of(kernel, threads, smem, a.rows, lanes() ? threads / std::max(1, lanes()) : 1, &grid)) return st;
        float *ws = nullptr;
        if (cudaMallocAsync(reinterpret_cast<void **>(&ws), size_t(grid) * 2 * a.dim * sizeof(float), s) != cudaSuccess) {
            cudaGetLastError();
            return int(SSM_ERR_CUDA);
        }
        a.part = ws;
        kernel<<<grid, threads, smem, s>>>(a);
        int st = status_of(cudaGetLastError());
        if (st == SSM_OK && (dw != nullptr || db != nullptr)) {
            ssm::layer_norm_cols_kernel<<<(2 * a.dim + 31) / 32, 256, 0, s>>>(ws, grid, a.dim, dw, db);
            st = status_of(cudaGetLastError());
        }
        const cudaError_t fe = cudaFreeAsync(ws, s);
        return st == SSM_OK && fe != cudaSuccess ? int(SSM_ERR_CUDA) : st;
    });
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

int ssm_layer_norm_bwd(const void *dy, const void *x, const float *weight, const float *mean,
                       const float *rstd, void *dx, float *dweight, float *dbias, int rows, int dim,
                       int in_dtype, int grad_dtype, void *cuda_stream) {
    if (!valid_dtype(in_dtype) || !valid_dtype(grad_dtype)) return SSM_ERR_INVALID_ARG;
    if (rows < 0 || dim < 1) return SSM_ERR_INVALID_ARG;
    if (dim > kMaxDim) return SSM_ERR_UNSUPPORTED;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return SSM_ERR_INVALID_ARG;
    for (const void *q : {dy, x, (const void *)weight, (const void *)mean, (const void *)rstd, (const void *)dx,
                          (const void *)dweight, (const void *)dbias})
        if (q && !aligned16(q)) return SSM_ERR_ALIGNMENT;
    const size_t n = size_t(rows) * dim, wb = size_t(dim) * 4, sb = size_t(rows) * 4, gb = n * dtype_size(grad_dtype);
    const struct { const void *p; size_t n; } in[] = {{x, n * dtype_size(in_dtype)}, {weight, wb}, {dy, gb}, {mean, sb}, {rstd, sb}};
    const struct { const void *p; size_t n; } out[] = {{dx, gb}, {dweight, wb}, {dbias, wb}};
    for (const auto &o : out) {
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
        return dim % 8 == 0 ? run_bwd<true, Ti, Tg>(a, dweight, dbias, s) : run_bwd<false, Ti, Tg>(a, dweight, dbias, s);
    });
}

}  // extern "C"
