// layer_norm.cuh -- layer norm over rows of `dim` values, and its backward.
//
//     y = (x - mean) rstd w + b,   mean = sum x / dim,   rstd = 1 / sqrt(sum (x - mean)^2 / dim + eps)
//     g = dy w,  xhat = (x - mean) rstd,  dx = rstd (g - mean(g) - xhat mean(g xhat))
//     dw = sum_rows dy xhat,  db = sum_rows dy
//
// Bound by HBM: a row is read once, kept in registers through its reductions (the variance
// from the centred values, all sums fp32) and written once.  A group of lanes owns a row: 8
// or 32 lanes of a warp for narrow rows, a CTA for wide ones, V vectors of 8 values each.
// Groups walk the rows with the grid's stride, their columns' weights in registers and the
// next row's loads in flight while the current one is reduced.  In the backward every lane
// also carries its columns' dw and db through its rows; the CTAs' sums go to scratch and a
// second kernel adds them in a fixed order (deterministic).
// Measured, bf16: 16384 rows of 768, 10.0 us (5.1 TB/s); 393216 rows of 64, 21.7 us (4.8 TB/s);
// backward of 16384 rows of 2560, 50 us (5.0 TB/s) and 6.7 us for the column sums.  Narrow rows
// are bound by their reductions' shuffles and the issue slots as much as by HBM.  The backward of
// wide rows off a multiple of 8 spills 44 to 64 bytes a thread.
#pragma once

#include "common.cuh"

namespace ssm {

struct NormArgs {
    const void *x, *dy;
    const float *w, *b;              // NULL: 1, 0
    void *out;                       // y, or dx
    float *mean, *rstd;              // forward: written (may be NULL); backward: read
    float *part;                     // backward: [CTAs][2][dim]
    long long rows;
    int dim;
    float eps;
};

// The lane's V vectors of 8 values of a row.  VEC (dim a multiple of 8, so that every row is
// 16-byte aligned): vector v is values 8 (v G + l) + 0..7.  Otherwise its values are G apart,
// one by one (a warp still covers whole lines).
template <int V, bool VEC> struct RowLanes {
    int l, G, dim;
    __device__ __forceinline__ int col(int v, int x) const { return VEC ? (v * G + l) * 8 + x : (v * 8 + x) * G + l; }
    __device__ __forceinline__ bool has(int v, int x) const { return col(v, VEC ? 0 : x) < dim; }

    template <typename T> __device__ __forceinline__ void load(const T *row, float (&f)[V][8], float fill) const {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (VEC) {
                if (has(v, 0)) {
                    load8<T>(row + col(v, 0), f[v]);
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x) f[v][x] = fill;
                }
            } else {
#pragma unroll
                for (int x = 0; x < 8; ++x) f[v][x] = has(v, x) ? to_f32(row[col(v, x)]) : fill;
            }
        }
    }
    template <typename T> __device__ __forceinline__ void store(T *row, const float (&f)[V][8]) const {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (VEC) {
                if (has(v, 0)) store8<T>(row + col(v, 0), f[v]);
            } else {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (has(v, x)) row[col(v, x)] = from_f32<T>(f[v][x]);
            }
        }
    }
};

// Raw bits of the next row, widened only when its turn comes (bf16 rows keep half the
// registers in flight).
template <int V, bool VEC, typename T> struct RawRow {
    static constexpr int W = sizeof(T) == 4 ? 8 : 4;      // words per vector
    uint32_t w[V][W];
    __device__ __forceinline__ void fetch(const T *row, const RowLanes<V, VEC> &r) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (VEC) {
                if (r.has(v, 0)) {
                    const uint4 *p = reinterpret_cast<const uint4 *>(row + r.col(v, 0));
#pragma unroll
                    for (int k = 0; k < W / 4; ++k) {
                        const uint4 q = __ldg(p + k);
                        w[v][4 * k] = q.x; w[v][4 * k + 1] = q.y; w[v][4 * k + 2] = q.z; w[v][4 * k + 3] = q.w;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < W; ++k) w[v][k] = 0;
                }
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    if constexpr (sizeof(T) == 4) {
                        w[v][k] = r.has(v, k) ? __float_as_uint(row[r.col(v, k)]) : 0u;
                    } else {
                        const uint16_t *h = reinterpret_cast<const uint16_t *>(row);
                        const uint32_t lo = r.has(v, 2 * k) ? h[r.col(v, 2 * k)] : 0u;
                        const uint32_t hi = r.has(v, 2 * k + 1) ? h[r.col(v, 2 * k + 1)] : 0u;
                        w[v][k] = lo | hi << 16;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void widen(float (&f)[V][8]) const {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                if constexpr (sizeof(T) == 4) f[v][x] = __uint_as_float(w[v][x]);
                else f[v][x] = __uint_as_float(x & 1 ? w[v][x >> 1] & 0xffff0000u : w[v][x >> 1] << 16);
            }
    }
};

// The sum of a value, or of a pair, over a group, to all of its lanes.  LANES = 8 or 32:
// shuffles; 0: the CTA, through shared memory, with two buffers in turn so that one barrier per
// sum is enough.
__device__ __forceinline__ float add_up(float a, float b) { return a + b; }
__device__ __forceinline__ float2 add_up(float2 a, float2 b) { return fadd2(a, b); }
__device__ __forceinline__ float shfl_xor(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ float2 shfl_xor(float2 v, int o) { return f2(shfl_xor(v.x, o), shfl_xor(v.y, o)); }
template <int LANES, typename T> __device__ __forceinline__ T group_sum(T v, float2 *sm, int &turn) {
#pragma unroll
    for (int o = (LANES == 8 ? 4 : 16); o > 0; o >>= 1) v = add_up(v, shfl_xor(v, o));
    if constexpr (LANES == 0) {
        T *buf = reinterpret_cast<T *>(sm + (turn & 1) * 32);
        ++turn;
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        const int nw = blockDim.x >> 5;
        v = T{};
        for (int w = 0; w < nw; ++w) v = add_up(v, buf[w]);
    }
    return v;
}

template <int LANES> struct NormGroups {
    long long first, stride;
    int l, G;
    __device__ __forceinline__ NormGroups() {
        if constexpr (LANES == 0) {
            first = blockIdx.x; stride = gridDim.x; l = threadIdx.x; G = blockDim.x;
        } else {
            const int per = blockDim.x / LANES;
            first = (long long)blockIdx.x * per + threadIdx.x / LANES;
            stride = (long long)gridDim.x * per;
            l = threadIdx.x % LANES; G = LANES;
        }
    }
};

// R rows per group and step (many narrow rows: more bytes in flight).  The arithmetic runs on packed
// pairs: with one value an instruction, rows of 64 were bound by issue (24.5 us for 393216).
template <int LANES, int V, int R, bool VEC, typename Tin, typename Tout>
__global__ void __launch_bounds__(LANES ? 256 : 512) layer_norm_fwd_kernel(const NormArgs p) {
    __shared__ float2 sm[64];
    const NormGroups<LANES> gr;
    const RowLanes<V, VEC> r{gr.l, gr.G, p.dim};
    const Tin *x = static_cast<const Tin *>(p.x);
    Tout *y = static_cast<Tout *>(p.out);
    RawRow<V, VEC, Tin> next[R];
    // whole warps walk the same number of steps (a narrow group past the end repeats row 0)
    const long long steps = (p.rows - gr.first + gr.stride * R - 1) / (gr.stride * R);
    const long long all = LANES == 8 ? (long long)__reduce_max_sync(0xffffffffu, unsigned(steps > 0 ? steps : 0))
                                     : (steps > 0 ? steps : 0);
    if (all == 0) return;
    auto fetch = [&](long long i) {
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const long long n = gr.first + (i * R + m) * gr.stride;
            next[m].fetch(x + size_t(n < p.rows ? n : 0) * p.dim, r);
        }
    };
    fetch(0);
    float w[V][8], b[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) { w[v][k] = 1.f; b[v][k] = 0.f; }
    if (p.w != nullptr) r.load(p.w, w, 0.f);
    if (p.b != nullptr) r.load(p.b, b, 0.f);
    const float inv = 1.f / float(p.dim);
    int turn = 0;
    for (long long i = 0; i < all; ++i) {
        float f[R][V][8];
#pragma unroll
        for (int m = 0; m < R; ++m) next[m].widen(f[m]);
        if (i + 1 < all) fetch(i + 1);
        float mean[R], rstd[R];
#pragma unroll
        for (int m = 0; m < R; ++m) {
            float2 s = f2(0.f, 0.f);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int k = 0; k < 8; k += 2) s = fadd2(s, f2(f[m][v][k], f[m][v][k + 1]));
            mean[m] = s.x + s.y;
        }
#pragma unroll
        for (int m = 0; m < R; ++m) mean[m] = group_sum<LANES>(mean[m], sm, turn) * inv;
#pragma unroll
        for (int m = 0; m < R; ++m) {
            float2 q = f2(0.f, 0.f);
            const float2 mm = f2(-mean[m], -mean[m]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float2 qv = f2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    float2 c = fadd2(f2(f[m][v][k], f[m][v][k + 1]), mm);
                    if constexpr (!VEC) {               // values past the row: nothing
                        if (!r.has(v, k)) c.x = 0.f;
                        if (!r.has(v, k + 1)) c.y = 0.f;
                    }
                    f[m][v][k] = c.x; f[m][v][k + 1] = c.y;
                    qv = ffma2(c, c, qv);
                }
                if (!VEC || r.has(v, 0)) q = fadd2(q, qv);
            }
            rstd[m] = q.x + q.y;
        }
#pragma unroll
        for (int m = 0; m < R; ++m) rstd[m] = 1.f / sqrtf(group_sum<LANES>(rstd[m], sm, turn) * inv + p.eps);
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const long long row = gr.first + (i * R + m) * gr.stride;
            const float2 rr = f2(rstd[m], rstd[m]);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    const float2 o = ffma2(fmul2(f2(f[m][v][k], f[m][v][k + 1]), rr), f2(w[v][k], w[v][k + 1]),
                                           f2(b[v][k], b[v][k + 1]));
                    f[m][v][k] = o.x; f[m][v][k + 1] = o.y;
                }
            if (row < p.rows) {
                r.store(y + size_t(row) * p.dim, f[m]);
                if (r.l == 0) {
                    if (p.mean != nullptr) p.mean[row] = mean[m];
                    if (p.rstd != nullptr) p.rstd[row] = rstd[m];
                }
            }
        }
    }
}

template <int LANES, int V, bool VEC, typename Tin, typename Tg>
__global__ void __launch_bounds__(LANES ? 256 : 512) layer_norm_bwd_kernel(const NormArgs p) {
    __shared__ float2 sm[64];
    extern __shared__ __align__(16) float cols[];          // LANES != 0: [2][dim]
    const NormGroups<LANES> gr;
    const RowLanes<V, VEC> r{gr.l, gr.G, p.dim};
    const Tin *x = static_cast<const Tin *>(p.x);
    const Tg *dy = static_cast<const Tg *>(p.dy);
    Tg *dx = static_cast<Tg *>(p.out);
    float dw[V][8], db[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[v][k] = db[v][k] = 0.f;
    const long long steps = (p.rows - gr.first + gr.stride - 1) / gr.stride;
    const long long all = LANES == 8 ? (long long)__reduce_max_sync(0xffffffffu, unsigned(steps > 0 ? steps : 0))
                                     : (steps > 0 ? steps : 0);
    auto row_of = [&](long long i) { const long long n = gr.first + i * gr.stride; return n < p.rows ? n : 0; };
    RawRow<V, VEC, Tin> nx;
    RawRow<V, VEC, Tg> ny;
    float nmean = 0.f, nrstd = 0.f, w[V][8];
    auto fetch = [&](long long i) {
        const long long row = row_of(i);
        nx.fetch(x + size_t(row) * p.dim, r);
        ny.fetch(dy + size_t(row) * p.dim, r);
        nmean = p.mean[row];
        nrstd = p.rstd[row];
    };
    if (all > 0) {
        fetch(0);
        if (p.w != nullptr) r.load(p.w, w, 0.f);
    }
    const float inv = 1.f / float(p.dim);
    int turn = 0;
    for (long long i = 0; i < all; ++i) {
        const long long row = row_of(i);
        const bool mine = gr.first + i * gr.stride < p.rows;
        float h[V][8], d[V][8];
        nx.widen(h);
        ny.widen(d);
        const float mean = nmean, rstd = nrstd;
        if (i + 1 < all) fetch(i + 1);
        float2 s = f2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                h[v][k] = r.has(v, k) ? (h[v][k] - mean) * rstd : 0.f;
                if (mine) {
                    dw[v][k] = fmaf(d[v][k], h[v][k], dw[v][k]);
                    db[v][k] += d[v][k];
                }
                if (p.w != nullptr) d[v][k] *= w[v][k];
                s.x += d[v][k];
                s.y = fmaf(d[v][k], h[v][k], s.y);
            }
        s = group_sum<LANES>(s, sm, turn);
        const float c1 = s.x * inv, c2 = s.y * inv;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int k = 0; k < 8; ++k) d[v][k] = rstd * (d[v][k] - fmaf(h[v][k], c2, c1));
        if (mine) r.store(dx + size_t(row) * p.dim, d);
    }
    // the CTA's column sums
    float *part = p.part + size_t(blockIdx.x) * 2 * p.dim;
    if constexpr (LANES == 0) {
        r.store(part, dw);
        r.store(part + p.dim, db);
    } else {
        if constexpr (LANES == 8) {
#pragma unroll
            for (int o = 8; o < 32; o <<= 1)
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        dw[v][k] += __shfl_xor_sync(0xffffffffu, dw[v][k], o);
                        db[v][k] += __shfl_xor_sync(0xffffffffu, db[v][k], o);
                    }
        }
        for (int t = 0; t < 8; ++t) {                       // warps in order
            if (int(threadIdx.x >> 5) == t && (threadIdx.x & 31) < LANES) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (r.has(v, k)) {
                            const int c = r.col(v, k);
                            cols[c] = (t ? cols[c] : 0.f) + dw[v][k];
                            cols[p.dim + c] = (t ? cols[p.dim + c] : 0.f) + db[v][k];
                        }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * p.dim; c += blockDim.x) part[c] = cols[c];
    }
}

// out[c] = sum over n parts of part[i][c], c < cols: 32 columns x 32 interleaved sums per CTA,
// added in a fixed order.  Columns below `dim` go to dw, the others to db.
__global__ void __launch_bounds__(1024) layer_norm_cols_kernel(const float *part, int n, int dim, float *dw, float *db) {
    __shared__ float sm[32][33];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
    float s = 0.f;
    if (c < 2 * dim)
#pragma unroll 8
        for (int i = ry; i < n; i += 32) s += part[size_t(i) * 2 * dim + c];
    sm[ry][cx] = s;
    __syncthreads();
    s = sm[cx][ry];                      // column ry's sums, one per lane
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int out = blockIdx.x * 32 + ry;
    if (cx == 0 && out < 2 * dim) {
        if (out < dim) { if (dw != nullptr) dw[out] = s; }
        else if (db != nullptr) db[out - dim] = s;
    }
}

}  // namespace ssm
