// Shared by the paged key-value cache's kernels: the device view of a cache and of an attention call, and host checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/q8_gemv.h"

namespace q8 {

void set_last_cuda_error(int e);  // q8_host.cpp

inline q8_status kv_cuda_fail(cudaError_t e) {
    set_last_cuda_error((int)e);
    return Q8_ERR_CUDA;
}
inline bool kv_aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool kv_overlap(const void *a, int64_t an, const void *b, int64_t bn) {
    return a && b && (uintptr_t)a < (uintptr_t)b + (uintptr_t)bn && (uintptr_t)b < (uintptr_t)a + (uintptr_t)an;
}
inline bool kv_is_q8(const q8_kv_cache *c) { return c->k_scale != nullptr; }
// Values from the first page's start to the last page's end.
inline int64_t kv_span(const q8_kv_cache *c) {
    return (int64_t)(c->pages - 1) * c->page_stride + (int64_t)c->heads * c->page_size * c->dim;
}
q8_status kv_check_cache(const q8_kv_cache *c);  // q8_kv.cu
bool kv_overlaps_cache(const q8_kv_cache *c, const void *p, int64_t bytes);

// One attention call (decode: row_start null, one row a request).
struct AttnArgs {
    const uint16_t *q;  // bf16 [rows][ldq]
    uint16_t *out;      // bf16 [rows][ldo]
    const void *k, *v;
    const float *ks, *vs;  // scales of a Q8_0 cache
    const int *table, *lens, *row_start;
    int64_t page_stride;  // values between pages
    int ldq, ldo;
    int pages, page_size, width, pitch;
    int rows, R, heads, kv_heads, group;  // group = heads / kv_heads
    float scale;
    int window, sinks;
    unsigned char *work;  // the caller's workspace
};

// Let `kernel` take `smem` bytes of dynamic shared memory, asked once a device: the attribute stays, and asking takes
// about as long as a launch.  `done` is the kernel's own, a bit a device.
template <typename Kernel>
inline cudaError_t kv_allow_smem(Kernel kernel, int smem, std::atomic<uint64_t> *done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launch with programmatic dependent launch: the kernel waits (griddepcontrol.wait) before it reads anything.
template <typename Kernel, typename... Args>
inline cudaError_t kv_launch(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace q8
