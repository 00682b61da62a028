// Linear layers with 4-bit weights and group scales. Format and contract: include/bitnet.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act_quant_device.cuh"
#include "bitnet_device.cuh"
#include "bitnet_internal.h"
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

// The forward. Bound by HBM: half a byte per weight, read once per tile of up to 32 tokens; the
// arithmetic is there to keep up with it (two weights per bf16 instruction, the products on
// mma.sync with 16 weight rows as its rows and 8 tokens as its columns, so one to eight tokens cost
// the same; tcgen05 has no use for 16-row tiles, and its operands would have to be unpacked into
// shared or tensor memory first).
//
// Rows are dealt out evenly, rows N c / G .. N (c + 1) / G to CTA c of G, in tiles of 16; the eight
// warps of a CTA take every eighth block of 128 weights of a tile (512 bytes of a row per step of
// the CTA) and add their sums in shared memory, in order. A warp's next P blocks (P KB) are
// always on their way in registers, across tiles, the first of them before the previous kernel
// of the stream has ended (weights do not depend on it).
constexpr int kW4Warps = kW4Threads / 32;
constexpr int kW4Pad = 20;  // floats per token in the reduction buffer: no bank conflicts

struct W4Params {
    const uint16_t* x;
    const uint8_t* packed;
    const uint16_t* scales;
    void* y;
    int64_t K, N, M;
    int32_t blocks;  // of 128 weights per row
    int32_t groups;  // scales per row
    int32_t out_f32;
};

__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Weights 2 i and 2 i + 1 of a word as a bf16 pair, exactly: 128 + code, less 136. The mask and
// the exponent go into one three-input logic instruction (written out: from C the compiler makes
// two, and the logic pipe is what comes next after HBM).
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i) {
    uint32_t v, r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(v)
        : "r"(word >> (4 * i)), "n"(0x000F000F), "r"(0x43004300));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x43084308u));
    return r;
}

__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: tiles of 8 tokens; NG: groups per block (1, 2 or 4); P: blocks in flight per warp.
template <int NT, int NG, int P>
__global__ void __launch_bounds__(kW4Threads, NT == 4 ? 1 : 2)
    linear_w4_kernel(const __grid_constant__ W4Params p) {
    __shared__ float red[2][kW4Warps][NT * 8 * kW4Pad];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int64_t r0 = p.N * blockIdx.x / gridDim.x, r1 = p.N * (blockIdx.x + 1) / gridDim.x;
    const int64_t m0 = int64_t(blockIdx.y) * (8 * NT);
    const int tiles = static_cast<int>((r1 - r0 + 15) / 16);
    const int mine = (p.blocks - warp + kW4Warps - 1) / kW4Warps;  // this warp's blocks of a tile
    const int64_t row_bytes = int64_t(p.blocks) * 64;

    uint4 wa[P], wb[P];
    uint32_t sa[P], sb[P];  // bf16 bits: scales of rows g and g + 8, of group c if NG > 1
    // Where the next block to load lies: this lane's 16 bytes of row g, and its scale.
    const int rows = static_cast<int>(r1 - r0);
    const uint8_t* wp = p.packed + (r0 + g) * row_bytes + warp * 64 + c * 16;
    const uint16_t* sp = p.scales + (r0 + g) * p.groups + warp * NG + (NG > 1 ? c : 0);
    const int64_t w8 = 8 * row_bytes, s8 = 8 * int64_t(p.groups);
    int left = mine;      // blocks of the tile to load
    int ra = g;           // row within the CTA's, `rows` and more behind the last tile
    int sg = warp * NG + (NG > 1 ? c : 0);
    auto load = [&](int i) {
        wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
        sa[i] = sb[i] = 0;
        const bool scaled = sg < p.groups && (NG != 2 || c < NG);
        if (ra < rows) {
            wa[i] = load_stream(wp);
            if (scaled) sa[i] = __ldg(sp);
        }
        if (ra + 8 < rows) {
            wb[i] = load_stream(wp + w8);
            if (scaled) sb[i] = __ldg(sp + s8);
        }
        wp += kW4Warps * 64;
        sp += kW4Warps * NG;
        sg += kW4Warps * NG;
        if (--left == 0) {
            left = mine;
            ra += 16;
            wp += 2 * w8 - mine * (kW4Warps * 64);
            sp += 2 * s8 - mine * (kW4Warps * NG);
            sg -= mine * (kW4Warps * NG);
        }
    };

    pdl_trigger();
    if (mine > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) load(i);
    }
    pdl_wait();

    float acc[NT][4] = {};
    int tile = 0, todo = mine;
    // This lane's x: token 8 t + g of the tile, 8 values of the block (zeros without a token).
    const uint16_t* xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t m = m0 + 8 * t + g;
        xp[t] = m < p.M ? p.x + m * p.K + warp * 128 + 8 * c : nullptr;
    }
    // The last block is half empty if K is not a multiple of 128; it falls to one warp.
    const bool cut = p.K % 128 != 0 && (p.blocks - 1) % kW4Warps == warp;
    auto finish = [&]() {  // a tile is done: the warps' sums, in order
        float* mybuf = red[tile & 1][warp];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mybuf[(8 * t + 2 * c + (e & 1)) * kW4Pad + g + 8 * (e >> 1)] = acc[t][e];
                acc[t][e] = 0.0f;
            }
        __syncthreads();  // (two buffers: the next tile writes the other one)
        for (int i = threadIdx.x; i < NT * 128; i += kW4Threads) {
            const int64_t m = m0 + (i >> 4), n = r0 + tile * 16 + (i & 15);
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kW4Warps; ++w) v += red[tile & 1][w][(i >> 4) * kW4Pad + (i & 15)];
            if (m < p.M && n < r1) {
                if (p.out_f32)
                    static_cast<float*>(p.y)[m * p.N + n] = v;
                else
                    static_cast<__nv_bfloat16*>(p.y)[m * p.N + n] = __float2bfloat16_rn(v);
            }
        }
        ++tile;
        todo = mine;
    };
    if (mine <= 0) {  // more warps than blocks: nothing to add
        while (tile < tiles) finish();
        return;
    }

    while (tile < tiles) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (tile < tiles) {
                const int64_t x0 = int64_t(mine - todo) * (kW4Warps * 128);
                const bool half = cut && todo == 1;
                float part[NT][4] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a = (&wa[i].x)[j], b = (&wb[i].x)[j];
                    const uint32_t a0 = w4_pair(a, 0), a1 = w4_pair(a, 1), a2 = w4_pair(a, 2),
                                   a3 = w4_pair(a, 3);
                    const uint32_t b0 = w4_pair(b, 0), b1 = w4_pair(b, 1), b2 = w4_pair(b, 2),
                                   b3 = w4_pair(b, 3);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        uint4 xv = make_uint4(0, 0, 0, 0);
                        if (xp[t] && !(j >= 2 && half))
                            xv = __ldg(reinterpret_cast<const uint4*>(xp[t] + x0 + 32 * j));
                        w4_mma(part[t], a0, b0, a1, b1, xv.x, xv.y);
                        w4_mma(part[t], a2, b2, a3, b3, xv.z, xv.w);
                    }
                    constexpr int kWords = 4 / NG;
                    if (j % kWords == kWords - 1) {  // a group ends
                        uint32_t fa = sa[i], fb = sb[i];
                        if (NG > 1) {
                            fa = __shfl_sync(0xFFFFFFFFu, fa, (lane & ~3) + j / kWords);
                            fb = __shfl_sync(0xFFFFFFFFu, fb, (lane & ~3) + j / kWords);
                        }
                        const float s0 = __uint_as_float(fa << 16), s1 = __uint_as_float(fb << 16);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            acc[t][0] += s0 * part[t][0];
                            acc[t][1] += s0 * part[t][1];
                            acc[t][2] += s1 * part[t][2];
                            acc[t][3] += s1 * part[t][3];
                            part[t][0] = part[t][1] = part[t][2] = part[t][3] = 0.0f;
                        }
                    }
                }
                load(i);
                if (--todo == 0) finish();
            }
        }
    }
}

template <int NT, int NG, int P>
cudaError_t launch_w4(const W4Params& p, cudaStream_t stream) {
    const int64_t tiles = (p.N + 15) / 16, most = int64_t(tc_num_sms()) * (NT == 4 ? 1 : 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles < most ? tiles : most),
                       static_cast<unsigned>((p.M + 8 * NT - 1) / (8 * NT)));
    cfg.blockDim = dim3(kW4Threads);
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_w4_kernel<NT, NG, P>, p);
}

template <int NG>
cudaError_t launch_w4_tokens(const W4Params& p, cudaStream_t stream) {
    if (p.M <= 8) return launch_w4<1, NG, 4>(p, stream);
    if (p.M <= 16) return launch_w4<2, NG, 3>(p, stream);
    return launch_w4<4, NG, 4>(p, stream);
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
    W4Params p = {x, packed, scales, y, K, N, M, static_cast<int32_t>((K + 127) / 128),
                  static_cast<int32_t>((K + group - 1) / group), out_f32};
    // 65535 token tiles of 32 per launch; a launch more only past two million tokens.
    constexpr int64_t kMost = 65535 * 32;
    for (int64_t m = 0; m < M; m += kMost) {
        p.x = x + m * K;
        p.y = static_cast<char*>(y) + m * N * (out_f32 ? 4 : 2);
        p.M = M - m < kMost ? M - m : kMost;
        const cudaError_t e = group == 128  ? launch_w4_tokens<1>(p, stream)
                              : group == 64 ? launch_w4_tokens<2>(p, stream)
                                            : launch_w4_tokens<4>(p, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace bitnet
