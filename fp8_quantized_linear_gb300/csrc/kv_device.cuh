// Pieces shared by the paged FP8 cache kernels: the cache's address
// arithmetic, the programmatic launch, the host checks of a cache.
#pragma once

#include <atomic>

#include "common.cuh"

namespace fp8l {

constexpr int64_t kKvMaxRequests = 8192;
constexpr float kKvMinScale = FP8L_KV_MIN_SCALE;  // of a page's block of keys or values

// Byte offset of token `o` (in its page), dimension 16 c of page-and-head
// `ph` = page * kv_heads + head: octets of tokens, then 16-byte chunks of
// dimensions, then the octet's eight rows.
__host__ __device__ __forceinline__ int64_t kv_chunk_offset(int64_t ph, int page_size, int dim, int o, int c) {
    return ph * page_size * dim + static_cast<int64_t>(o >> 3) * 8 * dim + c * 128 + (o & 7) * 16;
}

inline bool kv_page_size_ok(int64_t page_size) {
    return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128;
}

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Status of a CUDA call that failed.  The runtime keeps its error for the next
// look, which another entry point may take after a launch of its own: it is
// cleared here.
inline int cuda_failed() {
    (void)cudaGetLastError();
    return FP8L_ECUDA;
}

// Raises a kernel's shared-memory limit to `smem`, the most that any of its
// launches asks for, once per device (`ready` has a bit for each): a limit set
// for every launch could be lowered by another thread before the launch.
// `all_shared`: the SM's memory split in favour of shared memory.
template <typename Kernel>
inline int allow_smem(Kernel kernel, int smem, std::atomic<unsigned long long> &ready, bool all_shared) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cuda_failed();
    if (ready.load(std::memory_order_acquire) >> dev & 1u) return FP8L_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        (all_shared &&
         cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess))
        return cuda_failed();
    ready.fetch_or(1ull << dev, std::memory_order_release);
    return FP8L_OK;
}

// Launches `kernel` as a programmatic dependent of the preceding kernel on
// the stream: its blocks may become resident before that kernel ends, and
// run griddepcontrol.wait before their first global access.
template <typename Params>
inline int launch_dependent(void (*kernel)(Params), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                            const Params &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? FP8L_OK : cuda_failed();
}

// The larger one, NaN when either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ void grid_dependency_sync() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace fp8l
