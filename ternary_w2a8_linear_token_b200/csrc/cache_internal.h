// Internal declarations of the decode-step operators: 4-bit linear layers, the paged cache and
// attention over it.
#pragma once

#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "bitnet.h"

namespace bitnet {

// Launches under programmatic dependent launch: the kernel starts when its predecessor in the
// stream lets it or ends, and waits for the end (pdl_wait) before it touches what others may write.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                       cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Lets a kernel have up to `bytes` of dynamic shared memory on the current device, the same number
// on every call. `done` is the kernel's own: the devices on which that has been set, so that later
// calls do not ask the driver.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ----------------------------------------------------------------------------- 4-bit weights
__host__ __device__ inline int64_t w4_row_bytes(int64_t K) { return 64 * ((K + 127) / 128); }
cudaError_t launch_pack_w4(const float* W, int64_t N, int64_t K, int group, uint8_t* packed,
                           uint16_t* scales, cudaStream_t stream);
cudaError_t launch_linear_w4(const uint16_t* x, int64_t M, int64_t K, const uint8_t* packed,
                             const uint16_t* scales, int group, int64_t N, void* y, int out_f32,
                             cudaStream_t stream);

// ----------------------------------------------------------------------------- cache
// Most bytes a workspace of the upkeep calls needs for lists of n slots: a header, 8 bytes per
// page (two scratch words), 4 per slot (a mark) and 16 per list entry.
inline size_t cache_ws_bytes(int64_t num_pages, int64_t max_seqs, int64_t n) {
    return 256 + size_t(num_pages) * 8 + size_t(max_seqs) * 4 + size_t(n) * 16 + 256;
}

// The cache by value, as kernels take it.
struct CacheView {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    int32_t* error;
    int64_t max_pages;
    int32_t num_pages;
    int32_t max_seqs;
    int32_t kv_heads;
    int32_t page_shift;  // log2(page_size)
    int32_t head_dim;
    int32_t i8;
};

struct CacheLayers {
    bitnet_cache_layer layer[BITNET_CACHE_MAX_LAYERS];
};

cudaError_t launch_cache_fork(const CacheView& c, const int32_t* src, const int32_t* dst, int64_t n,
                              void* ws, cudaStream_t stream);
cudaError_t launch_cache_extend(const CacheView& c, const int32_t* seqs, const int32_t* add,
                                int64_t n, int32_t* copies, void* ws, cudaStream_t stream);
cudaError_t launch_cache_free(const CacheView& c, const int32_t* seqs, int64_t n, void* ws,
                              cudaStream_t stream);
cudaError_t launch_cache_compact(const CacheView& c, int32_t* copies, void* ws,
                                 cudaStream_t stream);
cudaError_t launch_cache_copy(const CacheView& c, const CacheLayers& layers, int nlayers,
                              const int32_t* copies, int64_t max_copies, cudaStream_t stream);
cudaError_t launch_cache_append(const CacheView& c, const bitnet_cache_layer& layer,
                                const uint16_t* k, const uint16_t* v, int64_t T,
                                const int32_t* seqs, const int32_t* pos, cudaStream_t stream);

// ----------------------------------------------------------------------------- attention
struct AttnParams {
    CacheView c;
    bitnet_cache_layer layer;
    const uint16_t* q;
    const int32_t* seqs;
    uint16_t* out;
    float* lse;
    void* ws;
    float scale;
    int32_t B;
    int32_t heads;
    int32_t window;  // 0: all positions
    int32_t sinks;
};
size_t attn_ws_bytes(int32_t head_dim);
cudaError_t launch_paged_attention(const AttnParams& p, cudaStream_t stream);

}  // namespace bitnet
