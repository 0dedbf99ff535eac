// api_scratch.cuh -- scratch memory and the wait counter for the entry points that need them.
#pragma once

#include "api_host.cuh"

namespace ssm_host {

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
