// Paged key/value cache: the write of new tokens and the upkeep of the pages (fork, extend with
// copy on write, free, compact, copy). Contracts: include/bitnet.h.
//
// Bookkeeping. refs alone says which pages are free, so there is no free list to keep in order:
// the pages that a call takes are the lowest-numbered free ones, whatever came before, and every
// result is a function of the tables (no atomic's order shows in it). A call that has to look at
// all of its list before it may change anything runs one CTA that validates and plans, then a
// grid that applies the plan; both read the list in order, so a failed check changes nothing.
#include <cuda_runtime.h>

#include "act_quant_device.cuh"
#include "cache_internal.h"

namespace bitnet {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kApplyChunk = 1024;  // table entries per CTA of an apply grid

// One list entry after planning.
struct Item {
    int32_t from;   // slot that is read, -1: skipped
    int32_t to;     // slot that is written
    int32_t pages;  // pages that `from` holds
    int32_t len;
};

// The workspace: a header, two words per page, one per slot, one Item per list entry.
struct Ws {
    int32_t* head;  // [0] 1 if the plan stands, [1] pages in use (compact)
    int32_t* a;     // (num_pages)
    int32_t* b;     // (num_pages)
    int32_t* mark;  // (max_seqs)
    Item* item;     // (n)
};

Ws ws_split(const CacheView& c, void* ws) {
    Ws w;
    w.head = static_cast<int32_t*>(ws);
    w.a = w.head + 64;
    w.b = w.a + c.num_pages;
    w.mark = w.b + c.num_pages;
    const uintptr_t end = reinterpret_cast<uintptr_t>(w.mark + c.max_seqs);
    w.item = reinterpret_cast<Item*>((end + 15) & ~uintptr_t(15));
    return w;
}

__device__ __forceinline__ int32_t pages_of(const CacheView& c, int32_t len) {
    return static_cast<int32_t>((int64_t(len) + (1 << c.page_shift) - 1) >> c.page_shift);
}

__device__ __forceinline__ bool len_fits(const CacheView& c, int64_t len) {
    return len >= 0 && len <= (c.max_pages << c.page_shift);
}

// Exclusive prefix sum over the CTA's threads (kPlanThreads of them); *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
    __shared__ int sums[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += up;
    }
    __syncthreads();  // the last call's reads of sums are done
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int s = sums[lane], all = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, all, d);
        if (lane >= d) all += up;
    }
    *total = __shfl_sync(0xFFFFFFFFu, all, 31);
    return inc - v + __shfl_sync(0xFFFFFFFFu, all - s, warp);
}

// Which of 32768 pages from `base` on are in use: this thread's word covers pages
// base + 32 * threadIdx.x + bit. Loads are coalesced (a warp reads 32 runs of 32 pages).
__device__ __forceinline__ uint32_t live_word(const CacheView& c, int64_t base) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = base + warp * 1024;
    int32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int64_t p = first + 32 * i + lane;
        r[i] = p < c.num_pages ? c.refs[p] : 1;
    }
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, r[i] != 0);
        if (lane == i) word = m;
    }
    return word;
}

// Marks every slot of a list and reports slots that are out of range or named twice. All threads
// of the CTA call it; *bad is shared and must be 0 on entry (and synchronised).
__device__ __forceinline__ void mark_slots(const CacheView& c, const Ws& w, const int32_t* also,
                                           const int32_t* seqs, int64_t n, int* bad) {
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t s = seqs[i];
        if (s < 0 || (also && also[i] < 0)) continue;
        if (s >= c.max_seqs || (also && also[i] >= c.max_seqs))
            atomicOr(bad, BITNET_CACHE_ERR_SEQ);
        else
            w.mark[s] = 0;
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t s = seqs[i];
        if (s < 0 || s >= c.max_seqs || (also && also[i] < 0)) continue;
        if (atomicAdd(&w.mark[s], 1) != 0) atomicOr(bad, BITNET_CACHE_ERR_SEQ);
    }
}

// Plans a fork (src given) or a free (src null): validates the list, then notes for each entry
// the slots, pages and length, so that the apply grid reads no length that it also writes.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(CacheView c, Ws w, const int32_t* src,
                                                            const int32_t* dst, int64_t n) {
    __shared__ int bad;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    mark_slots(c, w, src, dst, n, &bad);
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t to = dst[i], from = src ? src[i] : to;
        Item it = {-1, to, 0, 0};
        if (to >= 0 && from >= 0 && to < c.max_seqs && from < c.max_seqs) {
            if (src && c.lens[to] != 0) atomicOr(&bad, BITNET_CACHE_ERR_SEQ);
            it.len = c.lens[from];
            if (!len_fits(c, it.len)) {
                atomicOr(&bad, BITNET_CACHE_ERR_LEN);
            } else {
                it.from = from;
                it.pages = pages_of(c, it.len);
            }
        }
        w.item[i] = it;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        w.head[0] = bad == 0;
        if (bad) atomicOr(c.error, bad);
    }
}

// Applies a planned fork: blockIdx.x walks the pages of a row in chunks, blockIdx.y the list.
__global__ void __launch_bounds__(kApplyThreads) fork_kernel(CacheView c, Ws w, int64_t n) {
    if (!w.head[0]) return;
    for (int64_t i = blockIdx.y; i < n; i += gridDim.y) {
        const Item it = w.item[i];
        if (it.from < 0) continue;
        const int32_t* row = c.table + int64_t(it.from) * c.max_pages;
        int32_t* to = c.table + int64_t(it.to) * c.max_pages;
        for (int64_t j0 = int64_t(blockIdx.x) * kApplyChunk; j0 < it.pages;
             j0 += int64_t(gridDim.x) * kApplyChunk) {
#pragma unroll
            for (int u = 0; u < kApplyChunk / kApplyThreads; ++u) {
                const int64_t j = j0 + u * kApplyThreads + threadIdx.x;
                if (j >= it.pages) continue;
                const int32_t p = row[j];
                to[j] = p;
                if (uint32_t(p) < uint32_t(c.num_pages))
                    atomicAdd(&c.refs[p], 1);
                else
                    atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
            }
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) c.lens[it.to] = it.len;
    }
}

// Applies a planned free.
__global__ void __launch_bounds__(kApplyThreads) free_kernel(CacheView c, Ws w, int64_t n) {
    if (!w.head[0]) return;
    for (int64_t i = blockIdx.y; i < n; i += gridDim.y) {
        const Item it = w.item[i];
        if (it.from < 0) continue;
        const int32_t* row = c.table + int64_t(it.from) * c.max_pages;
        for (int64_t j0 = int64_t(blockIdx.x) * kApplyChunk; j0 < it.pages;
             j0 += int64_t(gridDim.x) * kApplyChunk) {
#pragma unroll
            for (int u = 0; u < kApplyChunk / kApplyThreads; ++u) {
                const int64_t j = j0 + u * kApplyThreads + threadIdx.x;
                if (j >= it.pages) continue;
                const int32_t p = row[j];
                if (uint32_t(p) < uint32_t(c.num_pages))
                    atomicSub(&c.refs[p], 1);
                else
                    atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
            }
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) c.lens[it.from] = 0;
    }
}

// Extend, in one CTA: validate, decide the copies on write, find the free pages, and only then
// change the tables. Bound by latency: the list is short (one entry per sequence of a batch), and
// 32768 reference counts are read per round until enough free ones are found.
__global__ void __launch_bounds__(kPlanThreads) extend_kernel(CacheView c, Ws w,
                                                              const int32_t* seqs,
                                                              const int32_t* add, int64_t n,
                                                              int32_t* copies) {
    __shared__ int bad;
    __shared__ unsigned long long want;  // pages that the call needs
    if (threadIdx.x == 0) {
        bad = 0;
        want = 0;
    }
    __syncthreads();
    const int32_t ps = 1 << c.page_shift;
    mark_slots(c, w, nullptr, seqs, n, &bad);
    // Item here: from = last page if it is shared and must not be written, else -1; to = slot
    // (-1: skipped); pages = pages held; len = length held.
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t s = seqs[i];
        Item it = {-1, -1, 0, 0};
        if (s >= 0 && s < c.max_seqs) {
            const int32_t len = c.lens[s], more = add[i];
            if (more < 0 || !len_fits(c, len) || !len_fits(c, int64_t(len) + more)) {
                atomicOr(&bad, BITNET_CACHE_ERR_LEN);
            } else {
                it.to = s;
                it.pages = pages_of(c, len);
                it.len = len;
                if (more > 0 && (len & (ps - 1)) != 0) {
                    const int32_t p = c.table[int64_t(s) * c.max_pages + it.pages - 1];
                    if (uint32_t(p) >= uint32_t(c.num_pages)) {
                        atomicOr(&bad, BITNET_CACHE_ERR_PAGE);
                    } else if (c.refs[p] > 1) {
                        it.from = p;
                        w.a[p] = 0;   // holders of p that grow in this call
                        w.b[p] = -1;  // the last of them
                    }
                }
            }
        }
        w.item[i] = it;
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0) {
            atomicOr(c.error, bad);
            copies[0] = 0;
            copies[1] = 0;
        }
        return;
    }
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t p = w.item[i].from;
        if (p < 0) continue;
        atomicAdd(&w.a[p], 1);
        atomicMax(&w.b[p], static_cast<int32_t>(i));
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        Item it = w.item[i];
        if (it.to < 0) continue;
        if (it.from >= 0 && w.a[it.from] == c.refs[it.from] && w.b[it.from] == i)
            w.item[i].from = it.from = -1;  // all holders grow, and this is the last: it keeps it
        const int32_t grown = pages_of(c, it.len + add[i]);
        atomicAdd(&want, static_cast<unsigned long long>(grown - it.pages + (it.from >= 0)));
    }
    __syncthreads();
    const int64_t total = static_cast<int64_t>(want);
    // The lowest `total` free pages, ascending, into a (the marks in a and b are done with).
    int64_t found = 0;
    for (int64_t base = 0; base < c.num_pages && found < total; base += 32768) {
        uint32_t word = ~live_word(c, base);
        int all;
        int64_t rank = found + block_scan(__popc(word), &all);
        found += all;
        const int32_t first = static_cast<int32_t>(base) + 32 * threadIdx.x;
        for (; word && rank < total; word &= word - 1) w.a[rank++] = first + __ffs(word) - 1;
    }
    if (found < total) {
        if (threadIdx.x == 0) {
            atomicOr(c.error, BITNET_CACHE_ERR_FULL);
            copies[0] = 0;
            copies[1] = 0;
        }
        return;
    }
    // Hand the pages out in list order: entry i takes the next (its copy first).
    int64_t page_base = 0;
    int copy_base = 0;
    for (int64_t i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int64_t i = i0 + threadIdx.x;
        Item it = {-1, -1, 0, 0};
        int need = 0, grown = 0;
        if (i < n) it = w.item[i];
        const bool cow = it.to >= 0 && it.from >= 0;
        if (it.to >= 0) {
            grown = pages_of(c, it.len + add[i]);
            need = grown - it.pages + cow;
        }
        int pages_all, copies_all;
        int64_t rank = page_base + block_scan(need, &pages_all);
        const int slot = copy_base + block_scan(cow, &copies_all);
        page_base += pages_all;
        copy_base += copies_all;
        if (it.to < 0) continue;
        int32_t* row = c.table + int64_t(it.to) * c.max_pages;
        if (cow) {
            const int32_t p = w.a[rank];
            copies[2 + 2 * int64_t(slot)] = it.from;
            copies[3 + 2 * int64_t(slot)] = p;
            atomicSub(&c.refs[it.from], 1);
        }
        for (int j = it.pages - cow; j < grown; ++j) {
            const int32_t p = w.a[rank++];
            row[j] = p;
            c.refs[p] = 1;
        }
        c.lens[it.to] = it.len + add[i];
    }
    if (threadIdx.x == 0) {
        copies[0] = copy_base;
        copies[1] = 0;
    }
}

// Compact, first step, in one CTA: with L pages in use, pairs the used pages from L on with the
// free ones below L, both ascending, moves their counts and leaves a[old] = new for the tables.
// a[k] (free pages) and a[old] do not meet: k < L <= old.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(CacheView c, Ws w,
                                                                    int32_t* copies) {
    int live = 0;
    for (int64_t base = 0; base < c.num_pages; base += 32768) {
        const int64_t first = base + 32 * threadIdx.x;
        const int64_t rest = c.num_pages - first;
        const uint32_t valid = rest >= 32 ? ~0u : rest <= 0 ? 0u : (1u << rest) - 1;
        int all;
        block_scan(__popc(live_word(c, base) & valid), &all);
        live += all;
    }
    int holes = 0, movers = 0;
    for (int64_t base = 0; base < c.num_pages; base += 32768) {
        const int32_t first = static_cast<int32_t>(base) + 32 * threadIdx.x;
        const int64_t rest = c.num_pages - first, low = int64_t(live) - first;
        const uint32_t valid = rest >= 32 ? ~0u : rest <= 0 ? 0u : (1u << rest) - 1;
        const uint32_t below = low >= 32 ? ~0u : low <= 0 ? 0u : (1u << low) - 1;
        const uint32_t word = live_word(c, base) & valid;
        uint32_t hole = ~word & valid & below, mover = word & ~below, dead = ~word & valid & ~below;
        int all;
        int rank = holes + block_scan(__popc(hole), &all);
        holes += all;
        for (; hole; hole &= hole - 1) w.a[rank++] = first + __ffs(hole) - 1;
        rank = movers + block_scan(__popc(mover), &all);
        movers += all;
        for (; mover; mover &= mover - 1) w.b[rank++] = first + __ffs(mover) - 1;
        for (; dead; dead &= dead - 1) w.a[first + __ffs(dead) - 1] = -1;  // nobody may hold it
    }
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += kPlanThreads) {
        const int32_t from = w.b[k], to = w.a[k];
        copies[2 + 2 * int64_t(k)] = from;
        copies[3 + 2 * int64_t(k)] = to;
        c.refs[to] = c.refs[from];
        c.refs[from] = 0;
        w.a[from] = to;
    }
    if (threadIdx.x == 0) {
        copies[0] = movers;
        copies[1] = 0;
        w.head[1] = live;
    }
}

// Compact, second step: the tables. blockIdx.x walks a row in chunks, blockIdx.y the slots.
__global__ void __launch_bounds__(kApplyThreads) compact_apply_kernel(CacheView c, Ws w) {
    const int32_t live = w.head[1];
    for (int64_t s = blockIdx.y; s < c.max_seqs; s += gridDim.y) {
        const int32_t len = c.lens[s];
        if (len == 0) continue;
        if (!len_fits(c, len)) {
            if (threadIdx.x == 0) atomicOr(c.error, BITNET_CACHE_ERR_LEN);
            continue;
        }
        const int32_t pages = pages_of(c, len);
        int32_t* row = c.table + s * c.max_pages;
        for (int64_t j0 = int64_t(blockIdx.x) * kApplyChunk; j0 < pages;
             j0 += int64_t(gridDim.x) * kApplyChunk) {
#pragma unroll
            for (int u = 0; u < kApplyChunk / kApplyThreads; ++u) {
                const int64_t j = j0 + u * kApplyThreads + threadIdx.x;
                if (j >= pages) continue;
                const int32_t p = row[j];
                const int32_t to = uint32_t(p) >= uint32_t(c.num_pages) ? -1
                                   : p < live                           ? p
                                                                        : w.a[p];
                if (to < 0)
                    atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
                else
                    row[j] = to;
            }
        }
    }
}

// Copies pages: the work is cut into pieces of 16 KB (256 threads x 4 x 16 bytes) over all pairs,
// layers and pools, and the grid strides over them. Bound by HBM: every byte read and written once.
constexpr int kCopyPieces = 4;
constexpr int64_t kCopyUnit = int64_t(kApplyThreads) * kCopyPieces * 16;

__global__ void __launch_bounds__(kApplyThreads) copy_kernel(CacheView c,
                                                             const __grid_constant__ CacheLayers l,
                                                             int nlayers, const int32_t* copies,
                                                             int64_t max_copies) {
    const int64_t tokens = int64_t(c.kv_heads) << c.page_shift;
    const int64_t data = tokens * c.head_dim * (c.i8 ? 1 : 2), scale = tokens * 4;
    const int64_t du = (data + kCopyUnit - 1) / kCopyUnit;
    const int64_t su = c.i8 ? (scale + kCopyUnit - 1) / kCopyUnit : 0;
    const int64_t per = 2 * (du + su) * nlayers;
    int64_t pairs = copies[0];
    if (pairs > max_copies) pairs = max_copies;
    for (int64_t unit = blockIdx.x; unit < pairs * per; unit += gridDim.x) {
        const int64_t pair = unit / per;
        int64_t r = unit - pair * per;
        const int li = static_cast<int>(r / (2 * (du + su)));
        r -= li * 2 * (du + su);
        const int32_t from = copies[2 + 2 * pair], to = copies[3 + 2 * pair];
        if (uint32_t(from) >= uint32_t(c.num_pages) || uint32_t(to) >= uint32_t(c.num_pages)) {
            if (threadIdx.x == 0) atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
            continue;
        }
        const bitnet_cache_layer& lay = l.layer[li];
        char* pool;
        int64_t bytes = data;
        if (r < 2 * du) {
            pool = static_cast<char*>(r < du ? lay.k : lay.v);
            if (r >= du) r -= du;
        } else {
            r -= 2 * du;
            bytes = scale;
            pool = reinterpret_cast<char*>(r < su ? lay.k_scale : lay.v_scale);
            if (r >= su) r -= su;
        }
        const uint4* in = reinterpret_cast<const uint4*>(pool + from * bytes);
        uint4* out = reinterpret_cast<uint4*>(pool + to * bytes);
        const int64_t pieces = bytes >> 4, p0 = r * (kCopyUnit >> 4) + threadIdx.x;
        uint4 v[kCopyPieces];
#pragma unroll
        for (int u = 0; u < kCopyPieces; ++u)
            if (p0 + u * kApplyThreads < pieces) v[u] = in[p0 + u * kApplyThreads];
#pragma unroll
        for (int u = 0; u < kCopyPieces; ++u)
            if (p0 + u * kApplyThreads < pieces) out[p0 + u * kApplyThreads] = v[u];
    }
}

// Writes new tokens. One thread per 8 values of a (token, pool, head) row, so D / 8 neighbouring
// lanes hold a row and its absolute maximum is a few shuffles away. Bound by HBM (K and V read
// once, pages written once), or by launch latency for one token per sequence.
template <int D>
__global__ void __launch_bounds__(kApplyThreads) append_kernel(CacheView c, bitnet_cache_layer lay,
                                                               const uint16_t* k,
                                                               const uint16_t* v, int64_t T,
                                                               const int32_t* seqs,
                                                               const int32_t* pos) {
    constexpr int kLanes = D / 8;
    const int64_t rows = 2 * T * c.kv_heads;
    const int64_t row = (int64_t(blockIdx.x) * kApplyThreads + threadIdx.x) / kLanes;
    const int piece = threadIdx.x % kLanes;
    if (row >= rows) return;  // kLanes neighbours leave together
    const bool is_v = row >= T * c.kv_heads;
    const int64_t r = is_v ? row - T * c.kv_heads : row;
    const int64_t t = r / c.kv_heads;
    const int head = static_cast<int>(r - t * c.kv_heads);
    const int64_t s = seqs ? seqs[t] : t;
    if (s < 0) return;
    if (s >= c.max_seqs) {
        if (piece == 0) atomicOr(c.error, BITNET_CACHE_ERR_SEQ);
        return;
    }
    const int32_t len = c.lens[s], at = pos ? pos[t] : len - 1;
    if (at < 0 || at >= len || !len_fits(c, len)) {
        if (piece == 0) atomicOr(c.error, BITNET_CACHE_ERR_LEN);
        return;
    }
    const int32_t page = c.table[s * c.max_pages + (at >> c.page_shift)];
    if (uint32_t(page) >= uint32_t(c.num_pages)) {
        if (piece == 0) atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
        return;
    }
    const uint4 x = reinterpret_cast<const uint4*>(is_v ? v : k)[r * kLanes + piece];
    const int64_t to = ((int64_t(page) * c.kv_heads + head) << c.page_shift) +
                       (at & ((1 << c.page_shift) - 1));
    if (!c.i8) {
        reinterpret_cast<uint4*>(is_v ? lay.v : lay.k)[to * kLanes + piece] = x;
        return;
    }
    // bf16 magnitudes order as unsigned integers: an exact maximum over the row's lanes.
    const uint32_t lanes = ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
    const float amax = bf16_lo(__reduce_max_sync(lanes, absmax8_bits(x)));
    const float scale = __fdiv_rn(127.0f, fmaxf(amax, kActEps));
    reinterpret_cast<uint2*>(is_v ? lay.v : lay.k)[to * kLanes + piece] = quant8(x, scale);
    if (piece == 0) (is_v ? lay.v_scale : lay.k_scale)[to] = scale;
}

dim3 apply_grid(const CacheView& c, int64_t rows) {
    const int64_t chunks = (c.max_pages + kApplyChunk - 1) / kApplyChunk;
    return dim3(static_cast<unsigned>(chunks < 64 ? chunks : 64),
                static_cast<unsigned>(rows < 4096 ? rows : 4096));
}

}  // namespace

cudaError_t launch_cache_fork(const CacheView& c, const int32_t* src, const int32_t* dst, int64_t n,
                              void* ws, cudaStream_t stream) {
    const Ws w = ws_split(c, ws);
    plan_kernel<<<1, kPlanThreads, 0, stream>>>(c, w, src, dst, n);
    fork_kernel<<<apply_grid(c, n), kApplyThreads, 0, stream>>>(c, w, n);
    return cudaGetLastError();
}

cudaError_t launch_cache_free(const CacheView& c, const int32_t* seqs, int64_t n, void* ws,
                              cudaStream_t stream) {
    const Ws w = ws_split(c, ws);
    plan_kernel<<<1, kPlanThreads, 0, stream>>>(c, w, nullptr, seqs, n);
    free_kernel<<<apply_grid(c, n), kApplyThreads, 0, stream>>>(c, w, n);
    return cudaGetLastError();
}

cudaError_t launch_cache_extend(const CacheView& c, const int32_t* seqs, const int32_t* add,
                                int64_t n, int32_t* copies, void* ws, cudaStream_t stream) {
    extend_kernel<<<1, kPlanThreads, 0, stream>>>(c, ws_split(c, ws), seqs, add, n, copies);
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CacheView& c, int32_t* copies, void* ws,
                                 cudaStream_t stream) {
    const Ws w = ws_split(c, ws);
    compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(c, w, copies);
    compact_apply_kernel<<<apply_grid(c, c.max_seqs), kApplyThreads, 0, stream>>>(c, w);
    return cudaGetLastError();
}

cudaError_t launch_cache_copy(const CacheView& c, const CacheLayers& layers, int nlayers,
                              const int32_t* copies, int64_t max_copies, cudaStream_t stream) {
    copy_kernel<<<148 * 8, kApplyThreads, 0, stream>>>(c, layers, nlayers, copies, max_copies);
    return cudaGetLastError();
}

cudaError_t launch_cache_append(const CacheView& c, const bitnet_cache_layer& layer,
                                const uint16_t* k, const uint16_t* v, int64_t T,
                                const int32_t* seqs, const int32_t* pos, cudaStream_t stream) {
    const int64_t threads = 2 * T * c.kv_heads * (c.head_dim / 8);
    const int64_t blocks = (threads + kApplyThreads - 1) / kApplyThreads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (c.head_dim == 64)
        append_kernel<64><<<static_cast<unsigned>(blocks), kApplyThreads, 0, stream>>>(
            c, layer, k, v, T, seqs, pos);
    else
        append_kernel<128><<<static_cast<unsigned>(blocks), kApplyThreads, 0, stream>>>(
            c, layer, k, v, T, seqs, pos);
    return cudaGetLastError();
}

}  // namespace bitnet
