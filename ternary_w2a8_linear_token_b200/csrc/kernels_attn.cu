// Attention of one new token per sequence over the paged cache. Contract: include/bitnet.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act_quant_device.cuh"
#include "cache_internal.h"

namespace bitnet {
namespace {

constexpr int kAttnThreads = 128;

// The operator, plainly: one CTA per (query, head), its warps take every fourth token, the lanes
// the dimensions; a running maximum and sum per warp, joined at the end.
template <int D>
__global__ void __launch_bounds__(kAttnThreads) attn_kernel(AttnParams p) {
    constexpr int E = D / 32;
    const CacheView& c = p.c;
    const int b = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kvh = h / (p.heads / c.kv_heads);
    const int64_t s = p.seqs ? p.seqs[b] : b;
    if (s < 0) return;
    if (s >= c.max_seqs) {
        if (threadIdx.x == 0) atomicOr(c.error, BITNET_CACHE_ERR_SEQ);
        return;
    }
    int64_t n = c.lens[s];
    const int64_t cap = c.max_pages << c.page_shift;
    if (n < 0 || n > cap) {
        if (threadIdx.x == 0) atomicOr(c.error, BITNET_CACHE_ERR_LEN);
        n = n < 0 ? 0 : cap;
    }
    const int64_t span = int64_t(p.window) + p.sinks;
    const int64_t seen = p.window && n > span ? span : n;
    float q[E], o[E] = {};
#pragma unroll
    for (int e = 0; e < E; ++e)
        q[e] = bf16_lo(p.q[(int64_t(b) * p.heads + h) * D + lane * E + e]);
    float top = -INFINITY, sum = 0.0f;
    for (int64_t i = warp; i < seen; i += kAttnThreads / 32) {
        const int64_t j = i < p.sinks ? i : i + (n - seen);
        const int32_t page = c.table[s * c.max_pages + (j >> c.page_shift)];
        if (uint32_t(page) >= uint32_t(c.num_pages)) {
            if (lane == 0) atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
            continue;
        }
        const int64_t row = ((int64_t(page) * c.kv_heads + kvh) << c.page_shift) +
                            (j & ((1 << c.page_shift) - 1));
        float k[E], v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t at = row * D + lane * E + e;
            if (c.i8) {
                k[e] = float(static_cast<const int8_t*>(p.layer.k)[at]) / p.layer.k_scale[row];
                v[e] = float(static_cast<const int8_t*>(p.layer.v)[at]) / p.layer.v_scale[row];
            } else {
                k[e] = bf16_lo(static_cast<const uint16_t*>(p.layer.k)[at]);
                v[e] = bf16_lo(static_cast<const uint16_t*>(p.layer.v)[at]);
            }
        }
        float z = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) z += q[e] * k[e];
#pragma unroll
        for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, d);
        z *= p.scale;
        const float next = fmaxf(top, z), keep = expf(top - next), w = expf(z - next);
        sum = sum * keep + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * v[e];
        top = next;
    }
    __shared__ float tops[4], sums[4], outs[4][D];
    if (lane == 0) {
        tops[warp] = top;
        sums[warp] = sum;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) outs[warp][lane * E + e] = o[e];
    __syncthreads();
    const float all = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    float total = 0.0f, f[4];
    for (int i = 0; i < 4; ++i) {
        f[i] = tops[i] == -INFINITY ? 0.0f : expf(tops[i] - all);
        total += f[i] * sums[i];
    }
    for (int d = threadIdx.x; d < D; d += kAttnThreads) {
        const float r = f[0] * outs[0][d] + f[1] * outs[1][d] + f[2] * outs[2][d] + f[3] * outs[3][d];
        p.out[(int64_t(b) * p.heads + h) * D + d] =
            __bfloat16_as_ushort(__float2bfloat16_rn(total > 0.0f ? r / total : 0.0f));
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[int64_t(b) * p.heads + h] = total > 0.0f ? all + logf(total) : -INFINITY;
}

}  // namespace

size_t attn_ws_bytes(int32_t, int32_t, int64_t, int64_t) { return 256; }

cudaError_t launch_paged_attention(const AttnParams& p, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.B), static_cast<unsigned>(p.heads));
    if (p.c.head_dim == 64)
        attn_kernel<64><<<grid, kAttnThreads, 0, stream>>>(p);
    else
        attn_kernel<128><<<grid, kAttnThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace bitnet
