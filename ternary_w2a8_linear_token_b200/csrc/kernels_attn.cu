// Attention of one new token per sequence over the paged cache. Contract: include/bitnet.h.
//
// Mathematics. For the query heads of one key/value head, with a running maximum m, sum l and
// weighted sum o per head (all binary32, base 2): for each tile of tokens
//   z = scale log2(e) q.k,  m' = max(m, max z),  p = 2^(z - m'),
//   l = l 2^(m - m') + sum p,  o = o 2^(m - m') + p v,  m = m',
// and two such states join by the same formula. out = o / l, lse = (m + log2 l) ln 2.
//
// Bound by HBM: every K and V byte is read once, for 2 to 32 multiply-adds. The products still run
// on the tensor cores (mma.sync m16n8k16, eight heads of a group as its columns), which leaves the
// issue slots to the loads; tcgen05 would need 64 rows and more to pay. p enters the second
// product as three bf16 terms, which hold all of its 24 bits, and a tile's products are summed from
// zero and added to o by rounded additions, since the tensor cores cut their sums off. Of 32768
// outputs (8 sequences of up to 65536 tokens, 8 bits) 8 then lie on the wrong side of a bf16 step,
// 22 in a plain binary32 form; with two terms and o as the products' accumulator it was 88, for 10 %
// less time in 8 bits (115 and 127 µs there) and 1 % in bf16 (137.0 and 138.5 µs, 48 sequences of up
// to 8192).
//
// Split. The tokens of all (sequence, key/value head, block of 16 heads) items are cut into units
// of 64 or 128, and every CTA takes an equal, contiguous share of all units, so that one long
// sequence among short ones keeps the whole GPU busy. The lengths are on the device, so each CTA
// finds its share there. A CTA's four warps take a quarter of each unit and load them through a ring
// of their own (cp.async, 16 bytes a lane, no barrier between warps); at the end of an item, or of
// the CTA's share, the four states are joined in shared memory, and the result goes out, or into
// the workspace if other CTAs hold parts of the item. A second kernel joins those, in order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "act_quant_device.cuh"
#include "bitnet_device.cuh"
#include "bitnet_internal.h"
#include "cache_internal.h"

namespace bitnet {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;         // heads per item
constexpr int kMinUnits = 2;      // fewest units that are worth a CTA of their own
constexpr int kJoinThreads = 128;
constexpr int kTerms = 3;     // bf16 terms of a weight: 24 bits, all that binary32 has
constexpr float kLag = 8.0f;  // powers of two that weights may exceed 1 by
// The maximum of scores that were all -inf or NaN: -inf itself stands for no visible token.
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A unit is kTile tokens for each warp: 16 of 256 bytes (a row of K or V), 32 of 128 or 64, so
// that a ring stage is 8 KB (4 KB for the smallest rows) and the work per tile that does not
// depend on its bytes weighs less. NH: blocks of eight heads in an item.
template <int D, bool I8, int NH>
struct Shape {
    static constexpr int kRowBytes = D * (I8 ? 1 : 2);
    static constexpr int kTile = kRowBytes == 256 ? 16 : 32;
    static constexpr int kUnit = kTile * kWarps;
    static constexpr int kPool = kTile * kRowBytes;  // K or V of one tile
    static constexpr int kStageBytes = 2 * kPool + (I8 ? 2 * kTile * 4 : 0);
    // CTAs per SM and stages of the ring: a third CTA where registers allow, with two stages for
    // rows of 128 bytes (D = 64 in bf16, 64 sequences in a window of 4100 tokens: 3.5 µs less than
    // with two CTAs of three stages; D = 128 in 8 bits, 8 sequences of up to 65536: 6 µs less).
    static constexpr int kCtas = D == 64 || (I8 && NH == 1) ? 3 : 2;
    static constexpr int kStages = kCtas == 3 && kRowBytes == 128 ? 2 : 3;
    // Shared memory in which the warps' states are joined.
    static constexpr int kJoinBytes = D == 128 && kCtas == 3 ? 4096 : 8192;
    static constexpr int kSmem = kWarps * kStages * kStageBytes + kJoinBytes;
};
constexpr int kMostCtas = 3;  // per SM, of any shape

// The workspace: the units and the CTAs that share them, a note of each CTA on the item that goes on
// behind its share, and two partial states per CTA.
struct Note {
    int32_t b;      // query of an item that begins in this share and ends in another, -1: none
    int32_t head0;  // first head
    int32_t rows;   // heads
    int32_t pad;
    int64_t end;    // last unit
};
struct AttnWs {
    int64_t* head;  // [0] CTAs, [1] units
    Note* note;     // [cta]
    float* part;    // [cta][2][kRows * D + 2 * kRows]: o, then m, then l
};

__host__ __device__ inline AttnWs attn_ws(void* ws, int most_ctas) {
    AttnWs w;
    w.head = static_cast<int64_t*>(ws);
    w.note = reinterpret_cast<Note*>(w.head + 32);
    w.part = reinterpret_cast<float*>(w.note + ((most_ctas + 15) & ~15));
    return w;
}

// Heads of a group in one item, and items of a sequence.
__host__ __device__ inline int head_blocks(int heads, int kv_heads) {
    return (heads / kv_heads + kRows - 1) / kRows;
}

// What a query sees: its slot (-1: none) and its visible tokens, of which those from the sinks on
// are shifted by `skip` positions.
struct Seen {
    int32_t slot, n, skip;
};

__device__ __forceinline__ Seen seen_by(const AttnParams& p, int64_t b, bool report) {
    const CacheView& c = p.c;
    Seen r = {-1, 0, 0};
    const int64_t s = p.seqs ? p.seqs[b] : b;
    if (s < 0) return r;
    if (s >= c.max_seqs) {
        if (report) atomicOr(c.error, BITNET_CACHE_ERR_SEQ);
        return r;
    }
    int64_t n = c.lens[s];
    const int64_t cap = c.max_pages << c.page_shift;
    if (n < 0 || n > cap) {
        if (report) atomicOr(c.error, BITNET_CACHE_ERR_LEN);
        n = n < 0 ? 0 : cap;
    }
    const int64_t span = int64_t(p.window) + p.sinks;
    const int64_t vis = p.window && n > span ? span : n;
    r.slot = static_cast<int32_t>(s);
    r.n = static_cast<int32_t>(vis);
    r.skip = static_cast<int32_t>(n - vis);
    return r;
}

// Units of one item of a query; a query without tokens still has one, which writes its zeros.
template <int UNIT>
__device__ __forceinline__ int32_t units_of(const Seen& s) {
    return s.slot < 0 ? 0 : s.n <= UNIT ? 1 : (s.n - 1) / UNIT + 1;
}

// a / b of non-negative numbers, in 32 bits where they fit: divisions of 64 bits were a tenth of a
// small call's time.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return uint32_t(a) / uint32_t(b);
    return a / b;
}
__device__ __forceinline__ int64_t share_begin(int64_t units, int64_t ctas, int64_t cta) {
    return quotient(units * cta, ctas);
}
__device__ __forceinline__ int64_t share_owner(int64_t units, int64_t ctas, int64_t unit) {
    return quotient((unit + 1) * ctas - 1, units);
}

struct Shared {
    Seen seen[kThreads];  // of the sequences from `base` on
    int64_t sums[kWarps], rest[kWarps];
    int64_t before;  // units before sequence `start`
    int32_t base, start;
    float m[kWarps][kRows], l[kWarps][kRows];
    uint32_t mask[kWarps][4];  // visible tokens of each ring stage
};

// A position in the list of units: sequence, then key/value head and block of its heads, then
// unit within that item.
struct Walk {
    int32_t b, head, block, t, units;
    Seen s;
};

template <int UNIT>
__device__ __forceinline__ void walk_enter(const AttnParams& p, const Shared& sh, Walk& w) {
    const uint32_t at = uint32_t(w.b - sh.base);
    w.s = at < uint32_t(kThreads) ? sh.seen[at] : seen_by(p, w.b, false);
    w.units = units_of<UNIT>(w.s);
}

// To the next unit; there must be one. (Where lengths change under the call there may be none: then
// the last query's come again, so that nothing is reached out of range.)
template <int UNIT>
__device__ __forceinline__ void walk_next(const AttnParams& p, const Shared& sh, int blocks,
                                          Walk& w) {
    if (++w.t < w.units) return;
    w.t = 0;
    if (++w.block < blocks) return;
    w.block = 0;
    if (++w.head < p.c.kv_heads) return;
    w.head = 0;
    do {
        if (w.b >= p.B - 1) break;
        ++w.b;
        walk_enter<UNIT>(p, sh, w);
    } while (w.units == 0);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Signed bytes 0 and 2 of w (odd: 1 and 3) as a bf16 pair, exactly: 128 + the low seven bits, less
// 128, or 256 for a negative byte (its sign bit is then the exponent's lowest). Two logic and one
// half-precision instruction for two values, the logic written out, since from C the compiler makes
// two of each; for V a form with one and three took 5 µs more (8 sequences of up to 65536 tokens, 32
// heads over 8). bf16 takes q as it is; K in fp16, with one permutation and one addition a pair, needs
// q scaled into fp16's range, where a head's small values lose bits, and took 127 µs where this takes
// 132 (16 sequences of 30000 over 2 heads: 93 and 91).
__device__ __forceinline__ uint32_t bytes_to_bf16(uint32_t w, bool odd) {
    if (odd) w >>= 8;
    uint32_t v, o, q;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "n"(0x007F007F), "r"(0x43004300));
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(o) : "r"(w), "n"(0x00800080), "r"(0x43004300));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(q) : "r"(v), "r"(o));
    return q;
}

// The 8 x 8 matrix of 16-bit values that the warp's registers hold, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// a, b -> their bf16 pair (a low), and what the rounding lost, exactly.
__device__ __forceinline__ uint32_t split_bf16(float& a, float& b) {
    uint32_t hi;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    a -= bf16_lo(hi);
    b -= bf16_hi(hi);
    return hi;
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a tile: chunks are permuted within 128
// bytes so that eight rows' equal chunks (one ldmatrix phase) lie in different banks.
template <int RB>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
    const int swz = RB == 64 ? (row >> 1) & 3 : row & 7;
    return uint32_t(row * RB + ((chunk ^ swz) << 4));
}

// Tokens (scores) and dimensions (output) are the rows of the products and heads their columns, so
// that up to eight heads cost one column block.
template <int D, bool I8, int NH>
__global__ void __launch_bounds__(kThreads, Shape<D, I8, NH>::kCtas)
    attn_kernel(const __grid_constant__ AttnParams p) {
    using Sh = Shape<D, I8, NH>;
    constexpr int RB = Sh::kRowBytes, S = Sh::kStages, T = Sh::kTile, UNIT = Sh::kUnit;
    constexpr int MT = T / 16;  // token tiles of sixteen
    constexpr uint32_t kAll = T == 32 ? ~0u : 0xFFFFu;  // mask of a full tile
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Shared sh;
    const CacheView& c = p.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = p.heads / c.kv_heads, blocks = head_blocks(p.heads, c.kv_heads);
    const int items = c.kv_heads * blocks;
    const AttnWs ws = attn_ws(p.ws, gridDim.x);

    pdl_wait();
    pdl_trigger();

    // This CTA's share of the units: their number first, then where the share begins. The first
    // sequences (all, in most batches) are looked at once for both.
    const Seen s0 = threadIdx.x < p.B ? seen_by(p, threadIdx.x, blockIdx.x == 0) : Seen{-1, 0, 0};
    auto scan = [&](int64_t v) {  // inclusive, within the warp
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= d) v += up;
        }
        return v;
    };
    int64_t mine = units_of<UNIT>(s0), upto = scan(mine), rest = 0;
    for (int64_t b = threadIdx.x + kThreads; b < p.B; b += kThreads)
        rest += units_of<UNIT>(seen_by(p, b, blockIdx.x == 0));
    if (p.B > kThreads) rest = __shfl_sync(0xFFFFFFFFu, scan(rest), 31);
    if (lane == 31) {
        sh.sums[warp] = upto;
        sh.rest[warp] = rest;
    }
    sh.seen[threadIdx.x] = s0;
    __syncthreads();
    int64_t all = 0;
    rest = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += sh.sums[w];
        all += sh.sums[w];
        rest += sh.rest[w];
    }
    const int64_t units = (all + rest) * items;
    const int64_t want = (units + kMinUnits - 1) / kMinUnits;
    const int64_t ctas = want < gridDim.x ? want : gridDim.x;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        ws.head[0] = ctas;
        ws.head[1] = units;
    }
    if (blockIdx.x >= ctas) return;
    const int64_t u0 = share_begin(units, ctas, blockIdx.x);
    const int64_t u1 = share_begin(units, ctas, int64_t(blockIdx.x) + 1);
    int64_t before = 0;
    for (int64_t b0 = 0;;) {
        const bool found = u0 < (before + all) * items;
        if (found) {
            if ((upto - mine) * items <= u0 && u0 < upto * items) {
                sh.before = (upto - mine) * items;
                sh.base = static_cast<int32_t>(b0);
                sh.start = static_cast<int32_t>(b0 + threadIdx.x);
            }
            break;
        }
        before += all;
        b0 += kThreads;
        if (b0 >= p.B) {  // no sequence holds u0: lengths have changed since the sum
            if (threadIdx.x == 0) ws.note[blockIdx.x].b = -1;
            return;
        }
        const int64_t next = b0 + threadIdx.x;
        const Seen s = next < p.B ? seen_by(p, next, false) : Seen{-1, 0, 0};
        mine = units_of<UNIT>(s);
        upto = scan(mine);
        __syncthreads();  // sums and seen have been read
        if (lane == 31) sh.sums[warp] = upto;
        sh.seen[threadIdx.x] = s;
        __syncthreads();
        all = 0;
        upto += before;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) upto += sh.sums[w];
            all += sh.sums[w];
        }
    }
    __syncthreads();

    Walk ahead;  // the unit whose pages are looked up next
    ahead.b = sh.start;
    walk_enter<UNIT>(p, sh, ahead);
    {
        const int64_t r = u0 - sh.before;
        const int32_t item = static_cast<int32_t>(quotient(r, ahead.units));
        ahead.t = static_cast<int32_t>(r - int64_t(item) * ahead.units);
        ahead.head = item / blocks;
        ahead.block = item - ahead.head * blocks;
    }
    Walk cur = ahead;
    // Units of this share: to do, to load, to look up (a share is below 2^31 units).
    const int32_t n_units = static_cast<int32_t>(u1 - u0);
    int32_t looked = 0, loaded = 0;

    uint8_t* ring = smem + warp * (S * Sh::kStageBytes);
    const uint32_t ring_at = smem_addr(ring);

    // Page lookup of one unit, a step ahead of its loads: lane i has token i (modulo T).
    int32_t row = 0;
    bool there = false;
    auto look_up = [&]() {
        if (looked >= n_units) return;
        const int32_t v = ahead.t * UNIT + warp * T + (lane & (T - 1));
        there = v < ahead.s.n;
        row = 0;
        if (there) {
            const int32_t j = v < p.sinks ? v : v + ahead.s.skip;
            const int32_t page =
                c.table[int64_t(ahead.s.slot) * c.max_pages + (j >> c.page_shift)];
            there = uint32_t(page) < uint32_t(c.num_pages);
            if (there)
                row = ((page * c.kv_heads + ahead.head) << c.page_shift) +
                      (j & ((1 << c.page_shift) - 1));
            else
                atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
        }
        if (++looked < n_units) walk_next<UNIT>(p, sh, blocks, ahead);
    };
    // Loads of the unit that was looked up last into a ring stage; one commit group per call, empty
    // behind the end.
    auto load = [&](int stage) {
        if (loaded < n_units) {
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there) & kAll;
            if (lane == 0) sh.mask[warp][stage] = mask;
            const uint32_t at = ring_at + stage * Sh::kStageBytes;
            constexpr int kLanes = RB / 16, kStep = 32 / kLanes;
            auto rows_in = [&](auto all) {
#pragma unroll
                for (int i = 0; i < T / kStep; ++i) {
                    const int r = i * kStep + lane / kLanes, ch = lane % kLanes;
                    const int64_t from =
                        int64_t(__shfl_sync(0xFFFFFFFFu, row, r)) * RB + ch * 16;
                    const bool ok = decltype(all)::value || (mask >> r & 1);
                    const uint32_t to = at + tile_at<RB>(r, ch);
                    cp_async16(to, static_cast<const uint8_t*>(p.layer.k) + from, ok);
                    cp_async16(to + Sh::kPool, static_cast<const uint8_t*>(p.layer.v) + from, ok);
                }
            };
            if (mask == kAll)
                rows_in(std::true_type());
            else
                rows_in(std::false_type());
            if (I8) {
                const uint32_t to = at + 2 * Sh::kPool + lane * 4;
                if (T == 32) {
                    cp_async4(to, p.layer.k_scale + row, there);
                    cp_async4(to + 4 * T, p.layer.v_scale + row, there);
                } else {
                    cp_async4(to, (lane < T ? p.layer.k_scale : p.layer.v_scale) + row, there);
                }
            }
            ++loaded;
        }
        cp_async_commit();
    };

    look_up();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        load(i);
        look_up();
    }

    const int g = lane >> 2, cq = lane & 3;
    uint32_t q[NH][D / 16][2];
    // o[h][i][e], m[h][e & 1], l[h][e & 1]: head 8 h + 2 cq + (e & 1), dimension dim_of(i, e >> 1).
    // m is the maximum that the sums stand on, which may lag behind by kLag (below).
    float o[NH][D / 16][4], m[NH][2], l[NH][2];
    auto dim_of = [&](int i, int half) { return 16 * i + (I8 ? 2 * g + half : g + 8 * half); };
    bool fresh = true;  // an item begins
    int stage = 0, rows = 0, head0 = 0;
    const float sc = p.scale * kLog2e;

    for (int32_t u = 0; u < n_units; ++u) {
        if (fresh) {
            fresh = false;
            rows = min(kRows, group - cur.block * kRows);
            head0 = cur.head * group + cur.block * kRows;
            const uint16_t* qb = p.q + (int64_t(cur.b) * p.heads + head0) * D;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const int r = 8 * h + g;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint2 w = make_uint2(0, 0);
                    const uint16_t* at = qb + r * D + 16 * ks;
                    if (r < rows) {
                        if (I8)
                            w = *reinterpret_cast<const uint2*>(at + 4 * cq);
                        else
                            w = make_uint2(*reinterpret_cast<const uint32_t*>(at + 2 * cq),
                                           *reinterpret_cast<const uint32_t*>(at + 8 + 2 * cq));
                    }
                    // in 8 bits pairs go in the order of the unpacked bytes
                    q[h][ks][0] = I8 ? __byte_perm(w.x, w.y, 0x5410) : w.x;
                    q[h][ks][1] = I8 ? __byte_perm(w.x, w.y, 0x7632) : w.y;
                }
                m[h][0] = m[h][1] = -INFINITY;
                l[h][0] = l[h][1] = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    o[h][i][0] = o[h][i][1] = o[h][i][2] = o[h][i][3] = 0.0f;
            }
        }

        cp_async_wait<S - 2>();
        __syncwarp();  // this unit's tile is in; all lanes are done with the last one
        load(stage == 0 ? S - 1 : stage - 1);
        look_up();

        const uint32_t mask = sh.mask[warp][stage];
        if (mask) {
            const uint32_t kt = ring_at + stage * Sh::kStageBytes, vt = kt + Sh::kPool;
            // One division per token: its factors replace its scales in shared memory (they are
            // read behind the products).
            float* scales =
                reinterpret_cast<float*>(ring + stage * Sh::kStageBytes + 2 * Sh::kPool);
            if (I8) {
                if (T == 32) {
                    scales[lane] = sc / scales[lane];
                    scales[T + lane] = 1.0f / scales[T + lane];
                } else {
                    scales[lane] = (lane < T ? sc : 1.0f) / scales[lane];
                }
                __syncwarp();
            }
            // z[h][t][2 half + e]: token 16 t + 8 half + g, head 8 h + 2 cq + e.
            float z[NH][MT][4];
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    z[h][t][0] = z[h][t][1] = z[h][t][2] = z[h][t][3] = 0.0f;
            const int lrow = lane & 15, lch = lane >> 4;
            if (I8) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ks += 2)
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        uint32_t r[4];
                        ldmatrix4(r, kt + tile_at<RB>(16 * t + lrow, ks + lch));
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t x = r[2 * k], y = r[2 * k + 1];
                            const uint32_t a[4] = {bytes_to_bf16(x, false), bytes_to_bf16(y, false),
                                                   bytes_to_bf16(x, true), bytes_to_bf16(y, true)};
#pragma unroll
                            for (int h = 0; h < NH; ++h)
                                mma_bf16(z[h][t], a, q[h][ks + k][0], q[h][ks + k][1]);
                        }
                    }
            } else {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        uint32_t a[4];
                        ldmatrix4(a, kt + tile_at<RB>(16 * t + lrow, 2 * ks + lch));
#pragma unroll
                        for (int h = 0; h < NH; ++h) mma_bf16(z[h][t], a, q[h][ks][0], q[h][ks][1]);
                    }
            }
            // Base-2 scores, less m. Hidden tokens get weight 0, and a factor that is not the
            // reciprocal of nothing.
            float f[MT][2], vs[MT][2], w[NH][MT][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    f[t][half] = I8 ? scales[16 * t + 8 * half + g] : sc;
                    if (I8) vs[t][half] = scales[T + 16 * t + 8 * half + g];
                }
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[h][t][x] = z[h][t][x] * f[t][x >> 1];
            if (mask != kAll) {
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        if (!(mask >> (16 * t + 8 * half + g) & 1)) {
                            vs[t][half] = 0.0f;
#pragma unroll
                            for (int h = 0; h < NH; ++h)
                                w[h][t][2 * half] = w[h][t][2 * half + 1] = -INFINITY;
                        }
            }
            bool grown = false;
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) m[h][e] = fmaxf(m[h][e], kLowest);
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int x = 0; x < 4; ++x) grown |= w[h][t][x] > m[h][x & 1] + kLag;
            // m follows the scores' maximum only when a weight would pass 2^kLag, so that most
            // tiles need neither the exchange between lanes nor a rescaling.
            if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = m[h][e];
#pragma unroll
                        for (int t = 0; t < MT; ++t)
                            top = fmaxf(top, fmaxf(w[h][t][e], w[h][t][2 + e]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                        const float keep = exp2_fast(m[h][e] - top);
                        m[h][e] = top;
                        l[h][e] *= keep;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            o[h][i][e] *= keep;
                            o[h][i][2 + e] *= keep;
                        }
                    }
            }
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int x = 2 * half + e;
                            w[h][t][x] = exp2_fast(w[h][t][x] - m[h][e]);
                            l[h][e] += w[h][t][x];
                        }
                }
            // Weights with tokens along the lanes' pairs, as the second product takes them.
            uint32_t term[MT][NH][kTerms][2];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float a = w[h][t][2 * half], b = w[h][t][2 * half + 1];
                        if (I8) {
                            a *= vs[t][half];
                            b *= vs[t][half];
                        }
#pragma unroll
                        for (int e = 0; e < kTerms; ++e)
                            term[t][h][e][half] = transpose8(split_bf16(a, b));
                    }
#pragma unroll
            for (int i = 0; i < D / 16; i += I8 ? 2 : 1) {
                float d[I8 ? 2 : 1][NH][4] = {};
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    uint32_t r[4];
                    if (I8)
                        ldmatrix4_trans(r, vt + tile_at<RB>(16 * t + lrow, i + lch));
                    else
                        ldmatrix4_trans(r, vt + tile_at<RB>(16 * t + (lane & 7) + (lane >> 4 << 3),
                                                            2 * i + (lane >> 3 & 1)));
#pragma unroll
                    for (int k = 0; k < (I8 ? 2 : 1); ++k) {
                        uint32_t a[4] = {r[0], r[1], r[2], r[3]};
                        if (I8) {
                            a[0] = bytes_to_bf16(r[2 * k], false);
                            a[1] = bytes_to_bf16(r[2 * k], true);
                            a[2] = bytes_to_bf16(r[2 * k + 1], false);
                            a[3] = bytes_to_bf16(r[2 * k + 1], true);
                        }
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int e = kTerms - 1; e >= 0; --e)
                                mma_bf16(d[k][h], a, term[t][h][e][0], term[t][h][e][1]);
                    }
                }
#pragma unroll
                for (int k = 0; k < (I8 ? 2 : 1); ++k)
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[h][i + k][x] += d[k][h][x];
            }
        }
        stage = stage + 1 == S ? 0 : stage + 1;

        if (cur.t + 1 == cur.units || u + 1 == n_units) {
            // Join the warps' states.
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
                        l[h][e] += __shfl_xor_sync(0xFFFFFFFFu, l[h][e], d);
                    if (g == 0) {
                        sh.m[warp][8 * h + 2 * cq + e] = m[h][e];
                        sh.l[warp][8 * h + 2 * cq + e] = l[h][e];
                    }
                }
            __syncthreads();
            float f[NH][2];
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * h + 2 * cq + e;
                    const float top =
                        fmaxf(fmaxf(sh.m[0][r], sh.m[1][r]), fmaxf(sh.m[2][r], sh.m[3][r]));
                    f[h][e] = exp2_fast(m[h][e] - (top == -INFINITY ? 0.0f : top));
                }
            const bool begun = u >= cur.t, ended = cur.t + 1 == cur.units;
            const bool whole = begun && ended;
            float* part = ws.part + (int64_t(blockIdx.x) * 2 + begun) * (kRows * D + 2 * kRows);
            // Columns go through shared memory in pieces that hold all warps' rows.
            float* buf = reinterpret_cast<float*>(smem + kWarps * S * Sh::kStageBytes);
            int piece = D;
            while (piece * rows * 4 * kWarps > Sh::kJoinBytes) piece >>= 1;
            for (int d0 = 0; d0 < D; d0 += piece) {
                if (d0) __syncthreads();
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 8 * h + 2 * cq + (e & 1), d = dim_of(i, e >> 1);
                            if (r < rows && d >= d0 && d < d0 + piece)
                                buf[(warp * rows + r) * piece + d - d0] = o[h][i][e] * f[h][e & 1];
                        }
                __syncthreads();
                for (int x = threadIdx.x; x < rows * piece; x += kThreads) {
                    const int r = x / piece, d = x - r * piece;
                    float v = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v += buf[(w * rows + r) * piece + d];
                    if (whole) {
                        float t = 0.0f;
                        const float b = fmaxf(fmaxf(sh.m[0][r], sh.m[1][r]),
                                              fmaxf(sh.m[2][r], sh.m[3][r]));
#pragma unroll
                        for (int w = 0; w < kWarps; ++w)
                            t += sh.l[w][r] * exp2_fast(sh.m[w][r] - b);
                        p.out[(int64_t(cur.b) * p.heads + head0 + r) * D + d0 + d] =
                            __bfloat16_as_ushort(
                                __float2bfloat16_rn(b == -INFINITY ? 0.0f : v / t));
                    } else {
                        part[r * D + d0 + d] = v;
                    }
                }
            }
            if (u + 1 == n_units && threadIdx.x == 0)
                ws.note[blockIdx.x] = {begun && !ended ? cur.b : -1, head0, rows, 0,
                                       u0 + u + (cur.units - 1 - cur.t)};
            if (threadIdx.x < rows) {
                const int r = threadIdx.x;
                const float b = fmaxf(fmaxf(sh.m[0][r], sh.m[1][r]), fmaxf(sh.m[2][r], sh.m[3][r]));
                const float base = b == -INFINITY ? 0.0f : b;
                float t = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) t += sh.l[w][r] * exp2_fast(sh.m[w][r] - base);
                if (!whole) {
                    part[kRows * D + r] = b;
                    part[kRows * D + kRows + r] = t;
                } else if (p.lse) {
                    p.lse[int64_t(cur.b) * p.heads + head0 + r] =
                        b == -INFINITY ? -INFINITY : (b + log2f(t)) * kLn2;
                }
            }
            __syncthreads();
            fresh = true;
        }
        if (u + 1 < n_units) walk_next<UNIT>(p, sh, blocks, cur);
    }
    cp_async_wait<0>();
}

// Joins the parts of the items that several CTAs worked on: blockIdx.x stands for a CTA of the
// split and takes head blockIdx.y of the item that goes on behind its share, if one does. A thread
// has four dimensions; groups of D / 4 threads take every n-th part, and their states join in a
// fixed order. Few CTAs have something to do, so they are small (64 sequences in a window of 4100
// tokens: 84 µs for both kernels, 87 with 256 threads, 97 with a CTA of 512 per query and head).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes, kAtOnce = 4;
    __shared__ float4 acc[kGroups][kLanes];
    __shared__ float tops[kGroups], sums[kGroups];
    pdl_wait();
    const AttnWs ws = attn_ws(p.ws, gridDim.x);
    const int c0 = blockIdx.x, r = blockIdx.y;
    const int64_t ctas = ws.head[0], units = ws.head[1];
    const Note note = ws.note[c0];  // (of a CTA without a share it says nothing)
    if (c0 >= ctas || note.b < 0 || r >= note.rows) return;
    // (beyond the CTAs only where lengths have changed under the call)
    const int last = static_cast<int>(min(share_owner(units, ctas, note.end), ctas - 1));
    const int grp = threadIdx.x / kLanes, d = threadIdx.x % kLanes;
    float top = -INFINITY, sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c1 = c0 + grp; c1 <= last; c1 += kAtOnce * kGroups) {
        float m[kAtOnce], l[kAtOnce];
        float4 v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int c = c1 + i * kGroups;
            m[i] = -INFINITY;
            l[i] = 0.0f;
            v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c > last) continue;
            // the item begins in c0's share and goes on in the others'
            const float* part = ws.part + (int64_t(c) * 2 + (c == c0)) * (kRows * D + 2 * kRows);
            m[i] = part[kRows * D + r];
            l[i] = part[kRows * D + kRows + r];
            v[i] = *reinterpret_cast<const float4*>(part + r * D + 4 * d);
        }
        float next = top;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) next = fmaxf(next, m[i]);
        const float base = next == -INFINITY ? 0.0f : next, a = exp2_fast(top - base);
        sum *= a;
        o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const float f = exp2_fast(m[i] - base);
            sum += l[i] * f;
            o.x += v[i].x * f;
            o.y += v[i].y * f;
            o.z += v[i].z * f;
            o.w += v[i].w * f;
        }
        top = next;
    }
    acc[grp][d] = o;
    if (d == 0) {
        tops[grp] = top;
        sums[grp] = sum;
    }
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) top = fmaxf(top, tops[i]);
    const float base = top == -INFINITY ? 0.0f : top;
    float total = 0.0f;
    o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const float f = exp2_fast(tops[i] - base);
        const float4 v = acc[i][d];
        total += sums[i] * f;
        o.x += v.x * f;
        o.y += v.y * f;
        o.z += v.z * f;
        o.w += v.w * f;
    }
    const float scale = top == -INFINITY ? 0.0f : 1.0f / total;  // (of no visible token: o is 0)
    const int64_t row = int64_t(note.b) * p.heads + note.head0 + r;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * scale, o.y * scale);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * scale, o.w * scale);
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * d) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (p.lse && d == 0) p.lse[row] = top == -INFINITY ? -INFINITY : (top + log2f(total)) * kLn2;
}

template <int D, bool I8, int NH>
cudaError_t launch_one(const AttnParams& p, cudaStream_t stream) {
    using Sh = Shape<D, I8, NH>;
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_smem(attn_kernel<D, I8, NH>, Sh::kSmem, allowed);
    if (e != cudaSuccess) return e;
    // CTAs of the split: as many as the GPU holds at once, whatever the lengths will be
    e = launch_pdl(attn_kernel<D, I8, NH>, dim3(tc_num_sms() * Sh::kCtas), kThreads, Sh::kSmem,
                   stream, p);
    if (e != cudaSuccess) return e;
    const int group = p.heads / p.c.kv_heads;
    return launch_pdl(join_kernel<D>, dim3(tc_num_sms() * Sh::kCtas, group < kRows ? group : kRows),
                      kJoinThreads, 0, stream, p);
}

template <int D, bool I8>
cudaError_t launch_groups(const AttnParams& p, cudaStream_t stream) {
    return p.heads / p.c.kv_heads > 8 ? launch_one<D, I8, 2>(p, stream)
                                      : launch_one<D, I8, 1>(p, stream);
}

}  // namespace

size_t attn_ws_bytes(int32_t head_dim) {
    const int most = tc_num_sms() * kMostCtas;
    return reinterpret_cast<size_t>(attn_ws(nullptr, most).part) +
           size_t(most) * 2 * (kRows * head_dim + 2 * kRows) * 4;
}

cudaError_t launch_paged_attention(const AttnParams& p, cudaStream_t stream) {
    if (p.c.head_dim == 64)
        return p.c.i8 ? launch_groups<64, true>(p, stream) : launch_groups<64, false>(p, stream);
    return p.c.i8 ? launch_groups<128, true>(p, stream) : launch_groups<128, false>(p, stream);
}

}  // namespace bitnet
