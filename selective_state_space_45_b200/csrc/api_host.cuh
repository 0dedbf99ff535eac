// api_host.cuh -- host-side argument helpers shared by the C ABI translation units.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/ssm.h"

namespace ssm_host {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_dtype(int t) { return t == SSM_F32 || t == SSM_BF16; }

inline int status_of(cudaError_t e) { return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA; }

inline size_t dtype_size(int t) { return t == SSM_F32 ? 4 : 2; }

// Do the byte ranges [p, p + pb) and [q, q + qb) share a byte?
inline bool overlaps(const void *p, size_t pb, const void *q, size_t qb) {
    if (!p || !q || pb == 0 || qb == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + qb && b < a + pb;
}

// Where kernels count the waits that they gave up on (ssm_device_timeouts reads it); NULL if it
// cannot be had on this device.
unsigned *wait_counter();

inline size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// A call's scratch: the caller's workspace if one is given, else a stream-ordered buffer
// that lives until release().
struct Scratch {
    unsigned char *p = nullptr;
    bool own = false;
    cudaStream_t s;
    int take(void *workspace, size_t given, size_t need, cudaStream_t stream) {
        s = stream;
        if (workspace) {
            if (given < need) return SSM_ERR_SCRATCH;
            p = static_cast<unsigned char *>(workspace);
            return SSM_OK;
        }
        if (cudaMallocAsync(reinterpret_cast<void **>(&p), need, s) != cudaSuccess) {
            cudaGetLastError();
            return SSM_ERR_CUDA;
        }
        own = true;
        return SSM_OK;
    }
    int release(int st) const {
        if (own && cudaFreeAsync(p, s) != cudaSuccess && st == SSM_OK) return SSM_ERR_CUDA;
        return st;
    }
};

}  // namespace ssm_host
