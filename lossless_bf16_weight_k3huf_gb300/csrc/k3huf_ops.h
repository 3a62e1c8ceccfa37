// Shared by the translation units of the operators that stand next to the
// coded weights (embedding rows, adapters, token log probabilities, products,
// control of logits, distillation): element loads and stores, warp sums,
// launches and argument checks.  Included from .cu files only.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "k3huf_internal.h"

namespace k3huf {

// --- device -----------------------------------------------------------------
__device__ __forceinline__ float ld_f32(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld_f32(const float *p) { return *p; }
// (one rounding, to nearest, at the end of an fp32 computation)
__device__ __forceinline__ void st_f32(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void st_f32(float *p, float v) { *p = v; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// A token id or adapter index of 4 or 8 bytes; negative ones mean "none".
__device__ __forceinline__ int64_t ld_id(const void *ids, uint32_t id_bytes, uint64_t i) {
    return id_bytes == 8 ? static_cast<const int64_t *>(ids)[i] : int64_t(static_cast<const int32_t *>(ids)[i]);
}

// The cluster's barrier in its two halves; the stores before the one are seen after the other.  (.aligned: a warp's threads
// come to it together, wherever they parted before.)
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// ... before which nothing is handed over (an exit: a release would wait for every store to memory)
__device__ __forceinline__ void cluster_arrive_relaxed() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// --- host -------------------------------------------------------------------
inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool elem_ok(uint32_t type) { return type == K3HUF_BF16 || type == K3HUF_F32; }
inline size_t elem_bytes(uint32_t type) { return type == K3HUF_F32 ? 4 : 2; }

// (the runtime's record of the error is cleared: the call returns it, nobody else should meet it)
inline int cuda_rc(cudaError_t e) {
    if (e == cudaSuccess) return K3HUF_OK;
    set_cuda_error(int(e));
    (void)cudaGetLastError();
    return K3HUF_E_CUDA;
}

// Runs f (a cudaFuncSetAttribute or the like) at a kernel's first launch on
// each device; two threads that do so at once set the same.
template <typename F>
int once_per_device(std::atomic<uint64_t> &done, F f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !((done.load(std::memory_order_acquire) >> dev) & 1))) {
        e = f();
        if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    }
    return cuda_rc(e);
}

// SMs of the current device.
inline int sm_count(uint64_t *sms) {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const bool kept = e == cudaSuccess && dev < 64;
    if (kept) n = known[dev].load(std::memory_order_relaxed);
    if (e == cudaSuccess && n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && kept) known[dev].store(n, std::memory_order_relaxed);
    }
    *sms = uint64_t(n > 0 ? n : 1);
    return cuda_rc(e);
}

}  // namespace k3huf
