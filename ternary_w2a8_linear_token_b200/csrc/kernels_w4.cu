// Linear layers with 4-bit weights and group scales. Format and contract: include/bitnet.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act_quant_device.cuh"
#include "cache_internal.h"

namespace bitnet {
namespace {

constexpr int kW4Threads = 256;

// Packs one block of 128 weights per 16 lanes: lane L holds the block's weights 8L .. 8L+7, which
// are one word of the format, and a group of 32, 64 or 128 weights is 4, 8 or 16 neighbouring
// lanes. Bound by HBM (the fp32 weights read once); off the per-token path.
__global__ void __launch_bounds__(kW4Threads) pack_w4_kernel(const float* __restrict__ W, int64_t N,
                                                             int64_t K, int group,
                                                             uint8_t* __restrict__ packed,
                                                             uint16_t* __restrict__ scales) {
    const int64_t blocks = (K + 127) / 128;
    const int64_t b = (int64_t(blockIdx.x) * kW4Threads + threadIdx.x) / 16;
    const int L = threadIdx.x & 15;
    if (b >= N * blocks) return;  // 16 neighbours leave together
    const int64_t n = b / blocks, kb = b - n * blocks;
    const int64_t k = kb * 128 + 8 * L;
    float w[8] = {};
    if (k < K) {  // K % 64 == 0: a lane is inside or outside as a whole
        const float4* p = reinterpret_cast<const float4*>(W + n * K + k);
        *reinterpret_cast<float4*>(w) = p[0];
        *reinterpret_cast<float4*>(w + 4) = p[1];
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(w[i]));
    const uint32_t lanes = 0xFFFFu << (threadIdx.x & 16);
    for (int d = 1; d < group / 8; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, d));
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(fmaxf(amax, 1e-5f), 7.0f));
    const float s = __bfloat162float(sb);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = fminf(fmaxf(rintf(__fdiv_rn(w[i], s)), -8.0f), 7.0f);
        word |= uint32_t(int(t) + 8) << (i & 1 ? 2 * i + 14 : 2 * i);
    }
    reinterpret_cast<uint32_t*>(packed)[b * 16 + 4 * (L & 3) + (L >> 2)] = word;
    if (k < K && k % group == 0)
        scales[n * ((K + group - 1) / group) + k / group] = __bfloat16_as_ushort(sb);
}

// The forward, plainly: one warp per weight row, a lane per word of 8 weights, one token after
// the other.
__global__ void __launch_bounds__(kW4Threads) linear_w4_kernel(
    const uint16_t* __restrict__ x, int64_t M, int64_t K, const uint8_t* __restrict__ packed,
    const uint16_t* __restrict__ scales, int group, int64_t N, void* __restrict__ y, int out_f32) {
    const int lane = threadIdx.x & 31;
    const int64_t n = int64_t(blockIdx.x) * (kW4Threads / 32) + (threadIdx.x >> 5);
    if (n >= N) return;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(packed + n * w4_row_bytes(K));
    const uint16_t* srow = scales + n * ((K + group - 1) / group);
    for (int64_t m = 0; m < M; ++m) {
        float acc = 0.0f;
        for (int64_t wd = lane; wd * 8 < w4_row_bytes(K) * 2; wd += 32) {
            const int64_t k = wd / 16 * 128 + wd % 4 * 32 + wd % 16 / 4 * 8;
            if (k >= K) continue;
            const uint32_t word = row[wd];
            const uint4 xv = *reinterpret_cast<const uint4*>(x + m * K + k);
            const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
            float part = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                part += bf16_lo(xs[i]) * float(int(word >> (4 * i) & 15) - 8);
                part += bf16_hi(xs[i]) * float(int(word >> (4 * i + 16) & 15) - 8);
            }
            acc += part * __uint_as_float(uint32_t(srow[k / group]) << 16);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, d);
        if (lane == 0) {
            if (out_f32)
                static_cast<float*>(y)[m * N + n] = acc;
            else
                static_cast<__nv_bfloat16*>(y)[m * N + n] = __float2bfloat16_rn(acc);
        }
    }
}

}  // namespace

cudaError_t launch_pack_w4(const float* W, int64_t N, int64_t K, int group, uint8_t* packed,
                           uint16_t* scales, cudaStream_t stream) {
    const int64_t blocks = (N * ((K + 127) / 128) * 16 + kW4Threads - 1) / kW4Threads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    pack_w4_kernel<<<static_cast<unsigned>(blocks), kW4Threads, 0, stream>>>(W, N, K, group, packed,
                                                                             scales);
    return cudaGetLastError();
}

cudaError_t launch_linear_w4(const uint16_t* x, int64_t M, int64_t K, const uint8_t* packed,
                             const uint16_t* scales, int group, int64_t N, void* y, int out_f32,
                             cudaStream_t stream) {
    linear_w4_kernel<<<static_cast<unsigned>((N + 7) / 8), kW4Threads, 0, stream>>>(
        x, M, K, packed, scales, group, N, y, out_f32);
    return cudaGetLastError();
}

}  // namespace bitnet
