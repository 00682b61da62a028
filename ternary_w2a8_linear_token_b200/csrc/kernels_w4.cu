// Linear layers with 4-bit weights and group scales. Format and contract: include/bitnet.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

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

// The forward. Bound by HBM: half a byte per weight, read once per 16 or 32 tokens; the
// arithmetic is there to keep up with it (two weights per bf16 instruction, the products on
// mma.sync with 16 weight rows as its rows and 8 tokens as its columns, so one to eight tokens cost
// the same; tcgen05 has no use for 16-row tiles, and its operands would have to be unpacked into
// shared or tensor memory first).
//
// A CTA is one or two teams of eight warps (one where two CTAs fit on an SM, so that the next
// call's can start as this one's end; two that share x where it takes more room). Rows are dealt
// out evenly over the teams, by 16 where each has more, and done in tiles of 16 RT; a team's warps
// take every eighth block of 128 weights of a tile (512 bytes of a row per step of the team) and
// add their sums in shared memory, in order. Every warp loads its blocks through a ring of its own
// (cp.async, no barrier between warps), across tiles, and fills it before the previous kernel of
// the stream has ended (weights do not depend on it). x and the scales come from shared memory:
// read by fragments from global memory, the eight rows of an instruction cost the L1 a tag lookup
// each.
constexpr int kW4Warps = 8;  // of a team
constexpr int kW4Teams = 2;  // most of a CTA, and of an SM
constexpr int kW4Stages = 4;
constexpr uint32_t kW4Room = 227 * 1024;  // shared memory of a CTA
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

// The same on zeros.
__device__ __forceinline__ void w4_mma_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Shared memory of a call: the rings, the teams' reduction buffers, two tiles' scales for each team
// as (group, row) with one row more, so that neither reads nor writes meet in a bank (those of a
// last, half block filled up with zeros), and x as (block, pair of tokens, quarter, token, 64
// bytes), zeros behind K: what a lane reads of either lies at fixed distances.
struct W4Layout {
    uint32_t red, scales, x, bytes;  // offsets; the rings come first
};
__host__ __device__ inline W4Layout w4_layout(int teams, int nt, int ng, int rt, int blocks,
                                              int tokens, bool xs) {
    W4Layout l;
    l.red = teams * kW4Warps * kW4Stages * rt * 1024;
    l.scales = l.red + teams * kW4Warps * nt * 8 * rt * kW4Pad * 4;
    l.x = l.scales + (teams * 2 * (16 * rt + 1) * 2 * blocks * ng + 15) / 16 * 16;
    l.bytes = l.x + (xs ? blocks * 512 * ((tokens + 1) / 2) : 0);
    return l;
}

// NT: tiles of 8 tokens; NG: groups per block (1, 2 or 4); RT: tiles of 16 rows that share a load
// of x; XS: x is in shared memory (otherwise read through L1).
template <int NT, int NG, int RT, bool XS>
__global__ void __launch_bounds__(32 * kW4Warps * kW4Teams, 1)
    linear_w4_kernel(const __grid_constant__ W4Params p) {
    constexpr int S = kW4Stages;
    constexpr int kRowsTile = 16 * RT;
    constexpr int kStage = RT * 1024;      // bytes of a block of a tile
    constexpr int kStep = kW4Warps * 64;   // bytes from one block of a warp to its next
    constexpr int kHeld = 4;               // scales per lane and row that are prefetched
    extern __shared__ __align__(128) uint8_t w4_dyn[];
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int team = threadIdx.x >> 8, warp = threadIdx.x >> 5 & (kW4Warps - 1);
    const int cta_teams = blockDim.x / (32 * kW4Warps);
    const int64_t teams = int64_t(gridDim.x) * cta_teams;
    const int64_t me = int64_t(blockIdx.x) * cta_teams + team;
    // Where a team has more than 16 rows, they begin at a multiple of 16 (a tile that is begun
    // costs as much as a full one: 14336 x 4096 at one token 10.7 against 11.0 µs).
    const int64_t deal = p.N > 16 * teams ? 16 : 1, deals = (p.N + deal - 1) / deal;
    const int64_t r0 = deals * me / teams * deal, r1 = min(deals * (me + 1) / teams * deal, p.N);
    const int64_t m0 = int64_t(blockIdx.y) * (8 * NT);
    const int tokens = static_cast<int>(p.M - m0 < 8 * NT ? p.M - m0 : 8 * NT);
    const int rows = static_cast<int>(r1 - r0), tiles = (rows + kRowsTile - 1) / kRowsTile;
    // This warp's blocks of a tile (a team may be without rows).
    const int mine = tiles ? (p.blocks - warp + kW4Warps - 1) / kW4Warps : 0;
    const int64_t row_bytes = int64_t(p.blocks) * 64;
    constexpr int kPitch = kRowsTile + 1;
    const int filled = p.blocks * NG;
    const int pair = 512 * ((tokens + 1) / 2);  // bytes of a block of x
    const W4Layout lay = w4_layout(cta_teams, NT, NG, RT, p.blocks, tokens, XS);
    float* const red = reinterpret_cast<float*>(w4_dyn + lay.red) +
                       team * (kW4Warps * NT * 8 * RT * kW4Pad);
    uint16_t* const scales = reinterpret_cast<uint16_t*>(w4_dyn + lay.scales) +
                             team * (2 * kPitch * filled);
    const uint8_t* const ring = w4_dyn + (team * kW4Warps + warp) * (S * kStage);
    const uint32_t ring_at = smem_addr(ring);

    // The blocks to load: tile, how many of it are left, and where this lane's 16 bytes of rows g,
    // g + 8, ... lie (rows behind the team's last repeat that one and are not written).
    int lt = 0, left = mine;
    const uint8_t* from[2 * RT];
    auto aim = [&]() {
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r)
            from[r] = p.packed + (r0 + min(lt * kRowsTile + 8 * r + g, rows - 1)) * row_bytes +
                      warp * 64 + c * 16;
    };
    auto load = [&](int i) {
        if (i < left) {
#pragma unroll
            for (int r = 0; r < 2 * RT; ++r)
                cp_async16(ring_at + i * kStage + (8 * r + g) * 64 + c * 16, from[r] + i * kStep,
                           true);
        }
        cp_async_commit();
    };
    auto advance = [&]() {  // past S blocks
        left -= S;
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) from[r] += S * kStep;
        if (left <= 0) {
            left = ++lt < tiles ? mine : 0;
            if (left > 0) aim();
        }
    };
    // Scales of a tile: a warp brings rows warp, warp + 8, ..., in registers until the tile before
    // it is done.
    uint16_t held[2 * RT][kHeld];
    auto scale_row = [&](int tile, int r) {
        return p.scales + (r0 + min(tile * kRowsTile + 8 * r + warp, rows - 1)) * p.groups;
    };
    auto fetch_scales = [&](int tile) {
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r)
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                held[r][i] =
                    32 * i + lane < p.groups ? __ldg(scale_row(tile, r) + 32 * i + lane) : 0;
    };
    auto store_scales = [&](int tile) {
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
            uint16_t* to = scales + (tile & 1) * (kPitch * filled) + 8 * r + warp;
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (32 * i + lane < filled) to[(32 * i + lane) * kPitch] = held[r][i];
            for (int i = 32 * kHeld + lane; i < filled; i += 32)
                to[i * kPitch] = i < p.groups ? __ldg(scale_row(tile, r) + i) : uint16_t(0);
        }
    };
    auto team_sync = [&]() {
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kW4Warps) : "memory");
    };

    pdl_trigger();
    if (tiles) {
        aim();
#pragma unroll
        for (int i = 0; i < S; ++i) load(i);
        advance();
        fetch_scales(0);
        store_scales(0);
    }
    pdl_wait();
    if (XS) {
        // Pieces of 8 values, U places of V tokens per thread on their way at once.
        auto bring = [&](auto u_, auto v_) {
            constexpr int U = decltype(u_)::value, V = decltype(v_)::value;
            const int places = p.blocks * 16, step = blockDim.x;
            for (int m1 = 0; m1 < tokens; m1 += V)
                for (int i0 = threadIdx.x; i0 < places; i0 += U * step) {
                    uint4 v[U][V];
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int m = 0; m < V; ++m) {
                            const int i = i0 + u * step;
                            v[u][m] = make_uint4(0, 0, 0, 0);
                            if (m1 + m < tokens && i < places && int64_t(i) * 8 < p.K)
                                v[u][m] = __ldg(reinterpret_cast<const uint4*>(
                                                    p.x + (m0 + m1 + m) * p.K) + i);
                        }
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int m = 0; m < V; ++m) {
                            const int i = i0 + u * step;
                            if (m1 + m < tokens && i < places)
                                *reinterpret_cast<uint4*>(
                                    w4_dyn + lay.x + (i >> 4) * pair + (m1 + m >> 1) * 512 +
                                    (i >> 2 & 3) * 128 + (m1 + m & 1) * 64 + (i & 3) * 16) =
                                    v[u][m];
                        }
                }
        };
        if (tokens == 1)
            bring(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
        else
            bring(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
    }
    __syncthreads();

    // This lane's x: token 8 t + g of the tile, 8 values of a quarter block. Columns behind the
    // last token repeat it and are not written.
    const uint8_t* xo[NT];
    const uint16_t* xg[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int m = min(8 * t + g, tokens - 1);
        xo[t] = w4_dyn + lay.x + warp * pair + (m >> 1) * 512 + (m & 1) * 64 + c * 16;
        xg[t] = p.x + (m0 + m) * p.K + warp * 128 + 8 * c;
    }
    // Without XS the last block's empty half is not read; it falls to one warp.
    const bool cut = !XS && p.K % 128 != 0 && (p.blocks - 1) % kW4Warps == warp;

    // One block of 128 weights by the tile's first R row tiles (the others have no rows).
    auto block = [&](auto R, const uint8_t* at, const uint16_t* sa, int xa, int64_t xv0, bool half,
                     float (&acc)[RT][NT][4]) {
        constexpr int kR = decltype(R)::value, kWords = 4 / NG;
        uint4 wa[kR], wb[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            wa[r] = *reinterpret_cast<const uint4*>(at + r * 1024);
            wb[r] = *reinterpret_cast<const uint4*>(at + r * 1024 + 512);
        }
        float part[kR][NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 xv[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                xv[t] = make_uint4(0, 0, 0, 0);
                if (XS)
                    xv[t] = *reinterpret_cast<const uint4*>(xo[t] + xa + j * 128);
                else if (j < 2 || !half)
                    xv[t] = __ldg(reinterpret_cast<const uint4*>(xg[t] + xv0 + 32 * j));
            }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const uint32_t a = (&wa[r].x)[j], b = (&wb[r].x)[j];
                const uint32_t a0 = w4_pair(a, 0), a1 = w4_pair(a, 1), a2 = w4_pair(a, 2),
                               a3 = w4_pair(a, 3);
                const uint32_t b0 = w4_pair(b, 0), b1 = w4_pair(b, 1), b2 = w4_pair(b, 2),
                               b3 = w4_pair(b, 3);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (j % kWords == 0)
                        w4_mma_new(part[r][t], a0, b0, a1, b1, xv[t].x, xv[t].y);
                    else
                        w4_mma(part[r][t], a0, b0, a1, b1, xv[t].x, xv[t].y);
                    w4_mma(part[r][t], a2, b2, a3, b3, xv[t].z, xv[t].w);
                }
                if (j % kWords == kWords - 1) {  // a group ends
                    const uint16_t* q = sa + 16 * r + j / kWords * kPitch;
                    const float s0 = __uint_as_float(uint32_t(q[0]) << 16);
                    const float s1 = __uint_as_float(uint32_t(q[8]) << 16);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        acc[r][t][0] += s0 * part[r][t][0];
                        acc[r][t][1] += s0 * part[r][t][1];
                        acc[r][t][2] += s1 * part[r][t][2];
                        acc[r][t][3] += s1 * part[r][t][3];
                    }
                }
            }
        }
    };

    for (int tile = 0; tile < tiles; ++tile) {
        if (tile + 1 < tiles) fetch_scales(tile + 1);
        const int below = min(rows - tile * kRowsTile, kRowsTile);  // rows of this tile
        float acc[RT][NT][4] = {};
        const uint16_t* sa = scales + (tile & 1) * (kPitch * filled) + warp * NG * kPitch + g;
        int xa = 0;  // bytes from the warp's first block of x to this one
        int64_t xv0 = 0;
        for (int todo = mine; todo > 0; todo -= S) {
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (i < todo) {
                    cp_async_wait<S - 1>();
                    __syncwarp();  // the block is in, from all lanes
                    const uint8_t* at = ring + i * kStage + g * 64 + c * 16;
                    const bool half = cut && i == todo - 1;
                    if (RT == 1 || below > 16)
                        block(std::integral_constant<int, RT>(), at, sa, xa, xv0, half, acc);
                    else
                        block(std::integral_constant<int, 1>(), at, sa, xa, xv0, half, acc);
                    __syncwarp();  // all lanes have read the stage
                }
                load(i);
                sa += kW4Warps * NG * kPitch;
                xa += kW4Warps * pair;
                xv0 += kW4Warps * 128;
            }
            advance();
        }
        // A tile is done: the warps' sums, in order.
        float* own = red + warp * (NT * 8 * RT * kW4Pad);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    own[((8 * t + 2 * c + (e & 1)) * RT + r) * kW4Pad + g + 8 * (e >> 1)] =
                        acc[r][t][e];
        if (tile + 1 < tiles) store_scales(tile + 1);
        team_sync();
        for (int i = threadIdx.x & (32 * kW4Warps - 1); i < NT * 8 * kRowsTile;
             i += 32 * kW4Warps) {
            const int m = i / kRowsTile, row = i % kRowsTile;
            const int64_t n = r0 + tile * kRowsTile + row;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kW4Warps; ++w)
                v += red[(w * (NT * 8) + m) * (RT * kW4Pad) + (row >> 4) * kW4Pad + (row & 15)];
            if (m < tokens && n < r1) {
                const int64_t to = (m0 + m) * p.N + n;
                if (p.out_f32)
                    static_cast<float*>(p.y)[to] = v;
                else
                    static_cast<__nv_bfloat16*>(p.y)[to] = __float2bfloat16_rn(v);
            }
        }
        team_sync();  // the buffer is free
    }
    cp_async_wait<0>();
}

// Without x the longest rows fit in every tile shape, in a CTA of one team.
static_assert(kW4Warps * kW4Stages * 2048 + kW4Warps * 8 * 2 * kW4Pad * 4 +
                      2 * 33 * 2 * BITNET_W4_MAX_GROUPS + 16 <= kW4Room &&
                  kW4Warps * kW4Stages * 1024 + kW4Warps * 32 * kW4Pad * 4 +
                          2 * 17 * 2 * BITNET_W4_MAX_GROUPS + 16 <= kW4Room,
              "the longest rows' scales fit beside the rings");

template <int NT, int NG, int RT, bool XS>
cudaError_t launch_w4_as(const W4Params& p, int teams, uint32_t smem, cudaStream_t stream) {
    auto kern = linear_w4_kernel<NT, NG, RT, XS>;
    static std::atomic<uint64_t> allowed;
    const cudaError_t e = allow_smem(kern, kW4Room, allowed);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.N + 15) / 16, ctas = int64_t(tc_num_sms()) * kW4Teams / teams;
    return launch_pdl(kern,
                      dim3(static_cast<unsigned>(tiles < ctas ? tiles : ctas),
                           static_cast<unsigned>((p.M + 8 * NT - 1) / (8 * NT))),
                      32 * kW4Warps * teams, smem, stream, p);
}

// x goes through shared memory where it fits: for one team on half an SM while a copy of x for
// each is small (one token of 14336 values, 4096 rows: 9.4 against 10.6 µs; 8 tokens of 4096
// values, 14336 rows: 12.3 against 11.7), for two on all of it otherwise.
template <int NT, int NG, int RT>
cudaError_t launch_w4(const W4Params& p, cudaStream_t stream) {
    const int tokens = static_cast<int>(p.M < 8 * NT ? p.M : 8 * NT);
    constexpr uint32_t kHalf = 113 * 1024, kCopy = 32 * 1024;
    const uint32_t one = w4_layout(1, NT, NG, RT, p.blocks, tokens, true).bytes;
    if (one <= kHalf && uint32_t(p.blocks) * 256 * tokens <= kCopy)
        return launch_w4_as<NT, NG, RT, true>(p, 1, one, stream);
    const uint32_t two = w4_layout(2, NT, NG, RT, p.blocks, tokens, true).bytes;
    if (two <= kW4Room) return launch_w4_as<NT, NG, RT, true>(p, 2, two, stream);
    return launch_w4_as<NT, NG, RT, false>(
        p, 1, w4_layout(1, NT, NG, RT, p.blocks, tokens, false).bytes, stream);
}

// The tile shape: 32 tokens a pass for up to 2^25 weights (6912 x 2560, 32 tokens: 11.4 µs against
// 13.0 in two passes of 16), 16 for more (28672 x 4096: 47 against 58; the second pass finds the
// weights in L2, and x takes half the reads); for up to eight tokens two row tiles share the reads
// of x where every team has more than one.
template <int NG>
cudaError_t launch_w4_tokens(const W4Params& p, cudaStream_t stream) {
    if (p.M > 16 && p.N * p.K <= int64_t(1) << 25) return launch_w4<4, NG, 1>(p, stream);
    if (p.M > 8) return launch_w4<2, NG, 1>(p, stream);
    if (p.N > 16 * kW4Teams * int64_t(tc_num_sms())) return launch_w4<1, NG, 2>(p, stream);
    return launch_w4<1, NG, 1>(p, stream);
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
    // 65535 token tiles of 16 or 32 per launch; a launch more only past a million tokens.
    constexpr int64_t kMost = 65535 * 16;
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
