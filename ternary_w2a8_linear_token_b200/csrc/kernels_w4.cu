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

// Behind the packing: a kernel that starts after the stores are visible. The forward reads weights and
// scales before its predecessor has ended, and so needs one that did not write them.
__global__ void w4_packed_kernel() {}

// The forward. Bound by HBM: half a byte per weight, read once per 16 or 32 tokens; the
// arithmetic is there to keep up with it (two weights per bf16 instruction, the products on
// mma.sync with 16 weight rows as its rows and 8 tokens as its columns, so one to eight tokens cost
// the same; tcgen05 has no use for 16-row tiles, and its operands would have to be unpacked into
// shared or tensor memory first).
//
// A CTA is eight warps where two CTAs fit on an SM, so that the next call's can start as this one's
// end, or sixteen that share x where it takes more room, in teams of W. Rows are dealt out evenly
// over the teams, by 16 where each has more, and done in tiles of 16 RT; a team's warps take every
// W-th block of 128 weights of a tile and add their sums in shared memory, in order. Every warp loads
// its blocks through a ring of its own (cp.async, no barrier between warps), across tiles, and fills
// it before the previous kernel of the stream has ended (weights do not depend on it). x and the
// scales come from shared memory: read by fragments from global memory, the eight rows of an
// instruction cost the L1 a tag lookup each.
//
// In bf16 a word's eight weights cost eleven instructions to unpack, and instructions, not HBM, bound
// large layers (131071 x 4096 at 68 % of the copy rate). Few tokens therefore go in bytes: x as
// 30-bit integers in units of 2^-28 of the largest value of a block, cut into four signed bytes, which
// take four of a product's columns; eight weights are then three instructions, the sums of a group
// are exact in 32-bit integers, and one subtraction makes a float of each (96 % there at one token).
// Values below 2^-20 of the largest lose bits, each at most 2^-29 of the largest. Binary32 sums lose
// as much where the largest value's product is among them, but nothing of the kind where its weight
// is 0 or its group's scale far below the others': there this form is the less exact one.
constexpr int kW4Most = 16;  // warps of a CTA, and of an SM
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

// Four of a word's eight weights as signed bytes 16 t: the high nibbles (words shifted left by 4:
// the low ones), in the order 2 6 3 7 (0 4 1 5). One mask and one change of the sign bit, in one
// logic instruction.
__device__ __forceinline__ uint32_t w4_bytes(uint32_t word) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(word), "n"(0xF0F0F0F0), "r"(0x80808080));
    return r;
}

__device__ __forceinline__ void w4_mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same on kW4Zero, whose bits are those of the float 1.5 * 2^23: sums v of less than 2^22 make
// it the float 1.5 * 2^23 + v, so that one subtraction turns them into floats.
constexpr int kW4Zero = 0x4B400000;
__device__ __forceinline__ void w4_mma_s8_new(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(kW4Zero));
}

// Eight values of x as 30-bit integers in units of 2^(E - 155) (E: the biased exponent of the
// largest of their block, at least 13), cut into four signed bytes each, of weights 1, 2^8, 2^15 and
// 2^23: to[128 d + half] (of odd d: to[128 d + 64 - half]) gets byte d of the values in the order of
// w4_bytes, low nibbles first.
__device__ __forceinline__ void w4_digits(const uint4& v, int E, uint8_t* to, int half) {
    // Adding 1.5 * 2^23 rounds to an integer and leaves it in the low bits; the 128 more carry what
    // makes the low byte signed, up to its sign bit.
    constexpr float kRound = 12582912.0f + 128.0f;
    const float scale = __uint_as_float(uint32_t(267 - E) << 23);
    uint32_t y[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = (&v.x)[i >> 1];
        const float h = (i & 1 ? bf16_hi(w) : bf16_lo(w)) * scale;  // below 2^14, exactly
        const float a = h + kRound;
        const float b = fmaf(h - (a - kRound), 32768.0f, kRound);  // of at most 2^14
        y[0][i] = __float_as_uint(b);
        y[1][i] = __float_as_uint(a);
    }
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const uint32_t a = __byte_perm(y[d][0], y[d][4], 0x5140);
        const uint32_t b = __byte_perm(y[d][1], y[d][5], 0x5140);
        const uint32_t e = __byte_perm(y[d][2], y[d][6], 0x5140);
        const uint32_t f = __byte_perm(y[d][3], y[d][7], 0x5140);
        *reinterpret_cast<uint2*>(to + d * 256 + half) =
            make_uint2(__byte_perm(a, b, 0x5410) ^ 0x80808080u,
                       __byte_perm(e, f, 0x5410) ^ 0x80808080u);
        *reinterpret_cast<uint2*>(to + d * 256 + 128 + 64 - half) =
            make_uint2(__byte_perm(a, b, 0x7632), __byte_perm(e, f, 0x7632));
    }
}

// Where x comes from: global memory through L1, shared memory, or shared memory as signed bytes
// (four columns of a product for each token, its four bytes).
enum W4X { kGlobal, kShared, kBytes };
__host__ __device__ constexpr int w4_tokens(W4X xm) { return xm == kBytes ? 2 : 8; }  // of a product

// Shared memory of a call: the rings, the teams' reduction buffers, two tiles' scales for each team
// as (group, row) with two rows more, so that neither reads nor writes meet in a bank, rows g and
// g + 8 of 16 next to each other (those of a last, half block filled up with zeros), and x, zeros
// behind K, as (block, pair of tokens, quarter, token, 64 bytes), or in bytes as (block, token, byte,
// half, c of a quarter, quarter, 8 bytes; of the odd bytes the second half first, against conflicts)
// and the units (block, token): what a lane reads of any lies at fixed distances.
struct W4Layout {
    uint32_t red, scales, x, units, bytes;  // offsets; the rings come first
};
__host__ __device__ inline W4Layout w4_layout(int warps, int teams, int nt, int ng, int rt,
                                              int blocks, int tokens, W4X xm) {
    W4Layout l;
    l.red = teams * warps * kW4Stages * rt * 1024;
    l.scales = l.red + teams * warps * nt * w4_tokens(xm) * rt * kW4Pad * 4;
    l.x = l.scales + (teams * 2 * (16 * rt + 2) * 2 * blocks * ng + 15) / 16 * 16;
    l.units = l.x + (xm == kBytes    ? blocks * 512 * tokens
                     : xm == kShared ? blocks * 512 * ((tokens + 1) / 2)
                                     : 0);
    l.bytes = l.units + (xm == kBytes ? blocks * tokens * 4 : 0);
    return l;
}

// NT: column tiles, of 8 tokens or of 2 in bytes; NG: groups per block (1, 2 or 4); RT: tiles of 16
// rows that share a load of x; XM: where x comes from; W: warps of a team.
template <int NT, int NG, int RT, W4X XM, int W>
__global__ void __launch_bounds__(32 * kW4Most, 1)
    linear_w4_kernel(const __grid_constant__ W4Params p) {
    constexpr int S = kW4Stages;
    constexpr int kRowsTile = 16 * RT;
    constexpr int kStage = RT * 1024;      // bytes of a block of a tile
    constexpr int kStep = W * 64;          // bytes from one block of a warp to its next
    constexpr int kMine = kRowsTile / W;   // rows whose scales a warp brings
    constexpr int kHeld = kMine < 4 ? 4 : 16 / kMine;  // per lane and row, prefetched
    constexpr int kTok = NT * w4_tokens(XM);
    extern __shared__ __align__(128) uint8_t w4_dyn[];
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int team = threadIdx.x / (32 * W), warp = threadIdx.x >> 5 & (W - 1);
    const int cta_teams = blockDim.x / (32 * W);
    const int64_t teams = int64_t(gridDim.x) * cta_teams;
    const int64_t me = int64_t(blockIdx.x) * cta_teams + team;
    // Where a team has more than 16 rows, they begin at a multiple of 16 (a tile that is begun
    // costs as much as a full one: 14336 x 4096 at one token 10.7 against 11.0 µs).
    const int64_t deal = p.N > 16 * teams ? 16 : 1, deals = (p.N + deal - 1) / deal;
    const int64_t r0 = deals * me / teams * deal, r1 = min(deals * (me + 1) / teams * deal, p.N);
    const int64_t m0 = int64_t(blockIdx.y) * kTok;
    const int tokens = static_cast<int>(p.M - m0 < kTok ? p.M - m0 : kTok);
    const int rows = static_cast<int>(r1 - r0), tiles = (rows + kRowsTile - 1) / kRowsTile;
    // This warp's blocks of a tile (a team may be without rows).
    const int mine = tiles ? (p.blocks - warp + W - 1) / W : 0;
    const int64_t row_bytes = int64_t(p.blocks) * 64;
    constexpr int kPitch = kRowsTile + 2;
    const int filled = p.blocks * NG;
    const int pair = 512 * (XM == kBytes ? tokens : (tokens + 1) / 2);  // bytes of a block of x
    const W4Layout lay = w4_layout(W, cta_teams, NT, NG, RT, p.blocks, tokens, XM);
    float* const red = reinterpret_cast<float*>(w4_dyn + lay.red) +
                       team * (W * kTok * RT * kW4Pad);
    uint16_t* const scales = reinterpret_cast<uint16_t*>(w4_dyn + lay.scales) +
                             team * (2 * kPitch * filled);
    const uint8_t* const ring = w4_dyn + (team * W + warp) * (S * kStage);
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
    // Scales of a tile: a warp brings rows warp, warp + W, ..., in registers until the tile before
    // it is done. Those of the first tile come from L2, as the rings' loads do: before the wait below L1
    // may hold what they were in an earlier call. (All of them from L2: 100000 x 4096 in groups of 32 at
    // 3 tokens 52.8 instead of 51.3 µs.)
    uint16_t held[kMine][kHeld];
    auto scale_row = [&](int tile, int r) {
        return p.scales + (r0 + min(tile * kRowsTile + W * r + warp, rows - 1)) * p.groups;
    };
    auto scale_at = [&](int tile, const uint16_t* at) { return tile ? __ldg(at) : __ldcg(at); };
    auto fetch_scales = [&](int tile) {
#pragma unroll
        for (int r = 0; r < kMine; ++r)
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                held[r][i] = 32 * i + lane < p.groups
                                 ? scale_at(tile, scale_row(tile, r) + 32 * i + lane)
                                 : 0;
    };
    auto store_scales = [&](int tile) {
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
            const int row = W * r + warp;
            uint16_t* to = scales + (tile & 1) * (kPitch * filled) + (row & 16) + 2 * (row & 7) +
                           (row >> 3 & 1);
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (32 * i + lane < filled) to[(32 * i + lane) * kPitch] = held[r][i];
            for (int i = 32 * kHeld + lane; i < filled; i += 32)
                to[i * kPitch] = i < p.groups ? scale_at(tile, scale_row(tile, r) + i) : uint16_t(0);
        }
    };
    auto team_sync = [&]() {
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * W) : "memory");
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
    if (XM != kGlobal) {
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
                            if (m1 + m >= tokens || i >= places) continue;
                            if (XM == kBytes) {
                                // 16 neighbours, alike in the conditions above, hold a block
                                const uint32_t top = __reduce_max_sync(
                                    0xFFFFu << (threadIdx.x & 16), absmax8_bits(v[u][m]));
                                const int E = max(int(top >> 7), 13);
                                const int at = (i >> 4) * tokens + m1 + m;
                                w4_digits(v[u][m], E,
                                          w4_dyn + lay.x + at * 512 + (i & 3) * 16 +
                                              (i >> 2 & 1) * 8,
                                          (i >> 3 & 1) * 64);
                                // 2^(E - 136), 2^23 / 16 of the unit (see the joining of the
                                // bytes' sums); NaN for a block with an Inf or NaN
                                if ((i & 15) == 0)
                                    reinterpret_cast<uint32_t*>(w4_dyn + lay.units)[at] =
                                        E == 255 ? 0x7FC00000u : uint32_t(E - 9) << 23;
                            } else {
                                *reinterpret_cast<uint4*>(
                                    w4_dyn + lay.x + (i >> 4) * pair + (m1 + m >> 1) * 512 +
                                    (i >> 2 & 3) * 128 + (m1 + m & 1) * 64 + (i & 3) * 16) =
                                    v[u][m];
                            }
                        }
                }
        };
        if (tokens == 1)
            bring(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
        else if (XM == kBytes && NT == 1)
            bring(std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
        else if (XM == kBytes)
            bring(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
        else
            bring(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
    }
    __syncthreads();

    // This lane's x: token 8 t + g of the tile, 8 values of a quarter block, or byte g % 4 of token
    // 2 t + g / 4, and the units of the columns that it holds sums of. Columns behind the last token
    // repeat it and are not written.
    const uint8_t* xo[NT];
    const uint16_t* xg[NT];
    const float* units[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (XM == kBytes) {
            xo[t] = w4_dyn + lay.x + warp * pair + min(2 * t + (g >> 2), tokens - 1) * 512 +
                    (g & 3) * 128 + (g & 1) * 64 + c * 16;
            units[t] = reinterpret_cast<const float*>(w4_dyn + lay.units) + warp * tokens +
                       min(2 * t + (c >> 1), tokens - 1);
            continue;
        }
        const int m = min(8 * t + g, tokens - 1);
        xo[t] = w4_dyn + lay.x + warp * pair + (m >> 1) * 512 + (m & 1) * 64 + c * 16;
        xg[t] = p.x + (m0 + m) * p.K + warp * 128 + 8 * c;
    }
    const int x_half = g & 1 ? -64 : 64;
    // In global memory the last block's empty half is not read; it falls to one warp.
    const bool cut = XM == kGlobal && p.K % 128 != 0 && (p.blocks - 1) % W == warp;

    // One block of 128 weights by the tile's first R row tiles (the others have no rows).
    auto block = [&](auto R, const uint8_t* at, const uint16_t* sa, int xa, int64_t xv0, bool half,
                     int ua, float (&acc)[RT][NT][4]) {
        constexpr int kR = decltype(R)::value, kWords = 4 / NG;
        uint4 wa[kR], wb[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            wa[r] = *reinterpret_cast<const uint4*>(at + r * 1024);
            wb[r] = *reinterpret_cast<const uint4*>(at + r * 1024 + 512);
        }
        if constexpr (XM == kBytes) {
            int part[kR][NT][4];
            uint4 xv[NT][2];
            float unit[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                xv[t][0] = *reinterpret_cast<const uint4*>(xo[t] + xa);
                xv[t][1] = *reinterpret_cast<const uint4*>(xo[t] + xa + x_half);
                unit[t] = units[t][ua];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const uint32_t a = (&wa[r].x)[j], b = (&wb[r].x)[j];
                    const uint32_t a0 = w4_bytes(a << 4), a1 = w4_bytes(b << 4),
                                   a2 = w4_bytes(a), a3 = w4_bytes(b);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4& x = xv[t][j >> 1];
                        const uint32_t b0 = j & 1 ? x.z : x.x, b1 = j & 1 ? x.w : x.y;
                        if (j % kWords == 0)
                            w4_mma_s8_new(part[r][t], a0, a1, a2, a3, b0, b1);
                        else
                            w4_mma_s8(part[r][t], a0, a1, a2, a3, b0, b1);
                    }
                    if (j % kWords == kWords - 1) {  // a group ends
                        const uint32_t q = *reinterpret_cast<const uint32_t*>(
                            sa + 16 * r + j / kWords * kPitch);
                        const float s0 = bf16_lo(q), s1 = bf16_hi(q);
                        const float zero = __int_as_float(kW4Zero);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const float q0 = s0 * unit[t], q1 = s1 * unit[t];
                            acc[r][t][0] += q0 * (__int_as_float(part[r][t][0]) - zero);
                            acc[r][t][1] += q0 * (__int_as_float(part[r][t][1]) - zero);
                            acc[r][t][2] += q1 * (__int_as_float(part[r][t][2]) - zero);
                            acc[r][t][3] += q1 * (__int_as_float(part[r][t][3]) - zero);
                        }
                    }
                }
            return;
        }
        float part[kR][NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 xv[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                xv[t] = make_uint4(0, 0, 0, 0);
                if (XM == kShared)
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
                    const uint32_t q = *reinterpret_cast<const uint32_t*>(
                        sa + 16 * r + j / kWords * kPitch);
                    const float s0 = bf16_lo(q), s1 = bf16_hi(q);
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
        const int next = tile + 1;
        if (next < tiles) {
            __builtin_assume(next > 0);
            fetch_scales(next);
        }
        const int below = min(rows - tile * kRowsTile, kRowsTile);  // rows of this tile
        float acc[RT][NT][4] = {};
        const uint16_t* sa = scales + (tile & 1) * (kPitch * filled) + warp * NG * kPitch + 2 * g;
        int xa = 0;  // bytes from the warp's first block of x to this one
        int64_t xv0 = 0;
        int ua = 0;
        for (int todo = mine; todo > 0; todo -= S) {
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (i < todo) {
                    cp_async_wait<S - 1>();
                    __syncwarp();  // the block is in, from all lanes
                    const uint8_t* at = ring + i * kStage + g * 64 + c * 16;
                    const bool half = cut && i == todo - 1;
                    if (RT == 1 || below > 16)
                        block(std::integral_constant<int, RT>(), at, sa, xa, xv0, half, ua,
                              acc);
                    else
                        block(std::integral_constant<int, 1>(), at, sa, xa, xv0, half, ua, acc);
                    __syncwarp();  // all lanes have read the stage
                }
                load(i);
                sa += W * NG * kPitch;
                xa += W * pair;
                xv0 += W * 128;
                ua += W * tokens;
            }
            advance();
        }
        // A tile is done: the warps' sums, in order.
        float* own = red + warp * (kTok * RT * kW4Pad);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (XM == kBytes) {
                    // Lanes of even c hold the sums of the bytes of weights 1 and 2^8, those of odd c
                    // of 2^15 and 2^23, all times 2^23: the largest is as large as the result.
                    const float f = c & 1 ? 0x1p-8f : 0x1p-23f;
                    float u0 = acc[r][t][0] * f + acc[r][t][1] * (256.0f * f);
                    float u1 = acc[r][t][2] * f + acc[r][t][3] * (256.0f * f);
                    u0 += __shfl_xor_sync(0xFFFFFFFFu, u0, 1);
                    u1 += __shfl_xor_sync(0xFFFFFFFFu, u1, 1);
                    float* to = own + ((2 * t + (c >> 1)) * RT + r) * kW4Pad + g;
                    if (!(c & 1)) {
                        to[0] = u0;
                        to[8] = u1;
                    }
                } else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    own[((8 * t + 2 * c + (e & 1)) * RT + r) * kW4Pad + g + 8 * (e >> 1)] =
                        acc[r][t][e];
        if (next < tiles) store_scales(next);
        team_sync();
        for (int i = threadIdx.x & (32 * W - 1); i < kTok * kRowsTile;
             i += 32 * W) {
            const int m = i / kRowsTile, row = i % kRowsTile;
            const int64_t n = r0 + tile * kRowsTile + row;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w)
                v += red[(w * kTok + m) * (RT * kW4Pad) + (row >> 4) * kW4Pad + (row & 15)];
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
static_assert(8 * kW4Stages * 2048 + 8 * 8 * 2 * kW4Pad * 4 +
                      2 * 34 * 2 * BITNET_W4_MAX_GROUPS + 16 <= kW4Room &&
                  8 * kW4Stages * 1024 + 8 * 32 * kW4Pad * 4 +
                          2 * 18 * 2 * BITNET_W4_MAX_GROUPS + 16 <= kW4Room,
              "the longest rows' scales fit beside the rings");

template <int NT, int NG, int RT, W4X XM, int W>
cudaError_t launch_w4_as(const W4Params& p, int teams, uint32_t smem, cudaStream_t stream) {
    constexpr int kTok = NT * w4_tokens(XM);
    auto kern = linear_w4_kernel<NT, NG, RT, XM, W>;
    static std::atomic<uint64_t> allowed;
    const cudaError_t e = allow_smem(kern, kW4Room, allowed);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.N + 15) / 16, ctas = int64_t(tc_num_sms()) * (kW4Most / W) / teams;
    return launch_pdl(kern,
                      dim3(static_cast<unsigned>(tiles < ctas ? tiles : ctas),
                           static_cast<unsigned>((p.M + kTok - 1) / kTok)),
                      32 * W * teams, smem, stream, p);
}

// x goes through shared memory where it fits (*fits): for eight warps on half an SM while a copy of
// x for each half is small (one token: 2560 x 2560 2.9 µs, on whole SMs 3.7; 28672 x 4096 13.2 and 13.7),
// for sixteen on all of it otherwise (14336 x 4096 at 8 tokens 10.7 µs, on halves 11.3; 4096 x 14336 at
// one 8.6 and 9.4).
template <int NT, int NG, int RT, W4X XM, int W>
cudaError_t launch_w4(const W4Params& p, bool* fits, cudaStream_t stream) {
    constexpr int kTok = NT * w4_tokens(XM), kTeams = kW4Most / W;
    const int tokens = static_cast<int>(p.M < kTok ? p.M : kTok);
    constexpr uint32_t kHalf = 113 * 1024, kCopy = 32 * 1024;
    const W4Layout half = w4_layout(W, kTeams / 2, NT, NG, RT, p.blocks, tokens, XM);
    const W4Layout whole = w4_layout(W, kTeams, NT, NG, RT, p.blocks, tokens, XM);
    *fits = true;
    if (half.bytes <= kHalf && half.bytes - half.x <= kCopy)
        return launch_w4_as<NT, NG, RT, XM, W>(p, kTeams / 2, half.bytes, stream);
    if (whole.bytes <= kW4Room)
        return launch_w4_as<NT, NG, RT, XM, W>(p, kTeams, whole.bytes, stream);
    *fits = false;
    return cudaSuccess;
}

// Where x does not fit beside two row tiles, one leaves it room (28672 x 4096, groups of 32, 8 tokens:
// 20.0 µs, and 24.6 with two tiles and x through L1).
template <int NT, int NG, int RT, int W>
cudaError_t launch_w4_bf16(const W4Params& p, cudaStream_t stream) {
    bool fits;
    cudaError_t e = launch_w4<NT, NG, RT, kShared, W>(p, &fits, stream);
    if constexpr (RT > 1)
        if (!fits) e = launch_w4<NT, NG, 1, kShared, W>(p, &fits, stream);
    if (fits) return e;
    return launch_w4_as<NT, NG, RT, kGlobal, 8>(
        p, 1, w4_layout(8, 1, NT, NG, RT, p.blocks, 0, kGlobal).bytes, stream);
}

// Few tokens go in bytes where the weights are many enough to pay for cutting x up (in bytes and in
// bf16, teams of eight): one token 2560 x 2560 3.3 and 3.0 µs, 2560 x 6912 4.7 and 4.9, 28672 x 4096
// 14.0 and 18.2, 131071 x 4096 45 and 63; two tokens 6912 x 2560 5.4 and 5.0, 14336 x 4096 9.2 and
// 10.8; three tokens, which take two column tiles, 14336 x 4096 11.2 and 10.9, 28672 x 4096 17.4 and
// 18.9, 131071 x 4096 55 and 64, but with groups of 64, and so more sums to turn into floats, 64 and
// 61.
template <int NG, int RT, int W>
cudaError_t launch_w4_few(const W4Params& p, cudaStream_t stream) {
    const int64_t weights = p.N * p.K;
    bool fits = false;
    cudaError_t e = cudaSuccess;
    if (p.M <= 2 && weights >= int64_t(1) << (p.M == 1 ? 24 : 25)) {
        e = launch_w4<1, NG, RT, kBytes, W>(p, &fits, stream);
        if (W < 8 && !fits) e = launch_w4<1, NG, RT, kBytes, 8>(p, &fits, stream);
    } else if constexpr (NG == 1) {
        if (p.M > 2 && p.M <= 4 && weights >= int64_t(1) << 26)
            e = launch_w4<2, NG, RT, kBytes, W>(p, &fits, stream);
    }
    return fits ? e : launch_w4_bf16<1, NG, RT, W>(p, stream);
}

// The tile shape: 32 tokens a pass for up to 2^25 weights (6912 x 2560, 32 tokens: 11.4 µs against
// 13.0 in two passes of 16), 16 for more (28672 x 4096: 47 against 58; the second pass finds the
// weights in L2, and x takes half the reads); for up to eight tokens two row tiles share the reads
// of x where every team has more than one. Teams of four warps where each has more than one tile
// and a tile's scales fit in registers: what a tile costs beside its blocks (scales, sums, barriers)
// then weighs half (teams of four and of eight: 10000 x 1024 4.1 and 4.7 µs, 131071 x 512 13.5 and
// 18.7, 14336 x 4096 at 8 tokens 10.5 and 11.7, at 16 13.2 and 14.3, 131071 x 4096 at 8 58 and 62;
// with too few rows 6912 x 2560 5.0 and 4.3).
template <int NG>
cudaError_t launch_w4_tokens(const W4Params& p, cudaStream_t stream) {
    if (p.M > 16 && p.N * p.K <= int64_t(1) << 25) return launch_w4_bf16<4, NG, 1, 8>(p, stream);
    const bool four = p.groups <= 64 && p.N > 64 * int64_t(tc_num_sms());
    if (p.M > 8)
        return four ? launch_w4_bf16<2, NG, 1, 4>(p, stream)
                    : launch_w4_bf16<2, NG, 1, 8>(p, stream);
    if (four) return launch_w4_few<NG, 2, 4>(p, stream);
    if (p.N > 32 * int64_t(tc_num_sms())) return launch_w4_few<NG, 2, 8>(p, stream);
    return launch_w4_few<NG, 1, 8>(p, stream);
}

}  // namespace

cudaError_t launch_pack_w4(const float* W, int64_t N, int64_t K, int group, uint8_t* packed,
                           uint16_t* scales, cudaStream_t stream) {
    const int64_t blocks = (N * ((K + 127) / 128) * 16 + kW4Threads - 1) / kW4Threads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    pack_w4_kernel<<<static_cast<unsigned>(blocks), kW4Threads, 0, stream>>>(W, N, K, group, packed,
                                                                             scales);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    w4_packed_kernel<<<1, 32, 0, stream>>>();
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
