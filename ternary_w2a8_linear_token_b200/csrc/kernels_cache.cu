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
#include "bitnet_device.cuh"
#include "bitnet_internal.h"
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
// base + 32 * threadIdx.x + bit, pages behind the pool in use. Loads are coalesced (a warp reads 32
// runs of 32 pages).
__device__ __forceinline__ uint32_t live_word(const CacheView& c, int64_t base) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = base + warp * 1024;
    const int rest = static_cast<int>(c.num_pages - first < 1024 ? c.num_pages - first : 1024);
    uint32_t word = ~0u;
    if (rest <= 0) return word;
    const int32_t* refs = c.refs + first + lane;
    int32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = 32 * i + lane < rest ? refs[32 * i] : 1;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, r[i] != 0);
        if (lane == i) word = m;
    }
    return word;
}

// Calls f(rank, page) for the pages that `word` (as live_word numbers them) names, this thread's
// first one being `rank`, ranks below `most`: a warp takes one word at a time, a lane per page, so
// that what f stores by rank or page lies together.
template <typename F>
__device__ __forceinline__ void for_pages(int64_t base, uint32_t word, int64_t rank, int64_t most,
                                          F f) {
    const int lane = threadIdx.x & 31;
    const int32_t first = static_cast<int32_t>(base) + (threadIdx.x >> 5) * 1024;
    if (!__any_sync(0xFFFFFFFFu, word != 0 && rank < most)) return;
#pragma unroll 4
    for (int i = 0; i < 32; ++i) {
        const uint32_t m = __shfl_sync(0xFFFFFFFFu, word, i);
        const int64_t r = __shfl_sync(0xFFFFFFFFu, rank, i) + __popc(m & ((1u << lane) - 1));
        if ((m >> lane & 1) && r < most) f(r, first + 32 * i + lane);
    }
}

// Marks every slot of a list and reports slots that are out of range or named twice: in a bitmap
// in shared memory, or for more slots than that holds in the workspace. All threads of the CTA
// call it; *bad is shared and must be 0 on entry (and synchronised).
constexpr int kMarkWords = 4096;
__device__ __forceinline__ void mark_slots(const CacheView& c, const Ws& w, const int32_t* also,
                                           const int32_t* seqs, int64_t n, int* bad) {
    __shared__ uint32_t bits[kMarkWords];
    const bool small = c.max_seqs <= 32 * kMarkWords;
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t s = seqs[i];
        if (s < 0 || (also && also[i] < 0)) continue;
        if (s >= c.max_seqs || (also && also[i] >= c.max_seqs))
            atomicOr(bad, BITNET_CACHE_ERR_SEQ);
        else if (small)
            bits[s >> 5] = 0;
        else
            w.mark[s] = 0;
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t s = seqs[i];
        if (s < 0 || s >= c.max_seqs || (also && also[i] < 0)) continue;
        const bool again = small ? atomicOr(&bits[s >> 5], 1u << (s & 31)) >> (s & 31) & 1
                                 : atomicAdd(&w.mark[s], 1) != 0;
        if (again) atomicOr(bad, BITNET_CACHE_ERR_SEQ);
    }
}

// Pages j of an entry of a fork: shared by one more slot.
__device__ __forceinline__ void fork_page(const CacheView& c, const Item& it, int64_t j) {
    const int32_t p = c.table[int64_t(it.from) * c.max_pages + j];
    c.table[int64_t(it.to) * c.max_pages + j] = p;
    if (uint32_t(p) < uint32_t(c.num_pages))
        atomicAdd(&c.refs[p], 1);
    else
        atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
}

// Pages j of an entry of a free: held by one slot less.
__device__ __forceinline__ void free_page(const CacheView& c, const Item& it, int64_t j) {
    const int32_t p = c.table[int64_t(it.from) * c.max_pages + j];
    if (uint32_t(p) < uint32_t(c.num_pages))
        atomicSub(&c.refs[p], 1);
    else
        atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
}

// Plans a fork (src given) or a free (src null): validates the list, then notes for each entry
// the slots, pages and length, so that what follows reads no length that it also writes. What
// follows is the apply grid, or with `alone` the same CTA, a warp per entry (see
// applies_alone).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(CacheView c, Ws w, const int32_t* src,
                                                            const int32_t* dst, int64_t n,
                                                            int alone) {
    __shared__ int bad;
    pdl_trigger();
    if (threadIdx.x == 0) bad = 0;
    pdl_wait();
    __syncthreads();
    mark_slots(c, w, src, dst, n, &bad);
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t to = dst[i], from = src ? src[i] : to;
        Item it = {-1, to, 0, 0};
        if (to >= 0 && from >= 0 && to < c.max_seqs && from < c.max_seqs) {
            const int32_t len = c.lens[from];
            if (src && c.lens[to] != 0) atomicOr(&bad, BITNET_CACHE_ERR_SEQ);
            if (!len_fits(c, len)) {
                atomicOr(&bad, BITNET_CACHE_ERR_LEN);
            } else {
                it.len = len;
                it.from = from;
                it.pages = pages_of(c, len);
            }
        }
        w.item[i] = it;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        w.head[0] = bad == 0;
        if (bad) atomicOr(c.error, bad);
    }
    if (!alone || bad) return;
    for (int64_t i = threadIdx.x >> 5; i < n; i += kPlanThreads / 32) {
        const Item it = w.item[i];
        if (it.from < 0) continue;
        for (int64_t j = threadIdx.x & 31; j < it.pages; j += 32) {
            if (src)
                fork_page(c, it, j);
            else
                free_page(c, it, j);
        }
        if ((threadIdx.x & 31) == 0) c.lens[it.to] = src ? it.len : 0;
    }
}

// Applies a planned fork or free: blockIdx.x walks the pages of a row in chunks, blockIdx.y the
// list.
template <bool FORK>
__global__ void __launch_bounds__(kApplyThreads) apply_kernel(CacheView c, Ws w, int64_t n) {
    pdl_trigger();
    pdl_wait();
    if (!w.head[0]) return;
    for (int64_t i = blockIdx.y; i < n; i += gridDim.y) {
        const Item it = w.item[i];
        if (it.from < 0) continue;
        for (int64_t j0 = int64_t(blockIdx.x) * kApplyChunk; j0 < it.pages;
             j0 += int64_t(gridDim.x) * kApplyChunk) {
#pragma unroll
            for (int u = 0; u < kApplyChunk / kApplyThreads; ++u) {
                const int64_t j = j0 + u * kApplyThreads + threadIdx.x;
                if (j >= it.pages) continue;
                if (FORK)
                    fork_page(c, it, j);
                else
                    free_page(c, it, j);
            }
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) c.lens[it.to] = FORK ? it.len : 0;
    }
}

// Extend, in one CTA: validate, decide the copies on write, find the free pages, and only then
// change the tables. Bound by latency: the list is short (one entry per sequence of a batch), and
// 32768 reference counts are read per round until enough free ones are found. ONE: at most one
// entry per thread, kept in registers between the steps instead of the workspace.
template <bool ONE>
__global__ void __launch_bounds__(kPlanThreads) extend_kernel(CacheView c, Ws w,
                                                              const int32_t* seqs,
                                                              const int32_t* add, int64_t n,
                                                              int32_t* copies) {
    __shared__ int bad;
    __shared__ long long wants[kPlanThreads / 32];
    pdl_trigger();
    if (threadIdx.x == 0) bad = 0;
    pdl_wait();
    __syncthreads();
    const int32_t ps = 1 << c.page_shift;
    mark_slots(c, w, nullptr, seqs, n, &bad);
    // Item here: from = last page if it is shared and must not be written, else -1; to = slot
    // (-1: skipped); pages = pages held; len = length held.
    Item own = {-1, -1, 0, 0};
    int32_t own_add = 0;
    auto item = [&](int64_t i) { return ONE ? own : w.item[i]; };
    auto more = [&](int64_t i) { return ONE ? own_add : add[i]; };
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        const int32_t s = seqs[i], grow = add[i];
        Item it = {-1, -1, 0, 0};
        if (s >= 0 && s < c.max_seqs) {
            const int32_t len = c.lens[s];
            if (grow < 0 || !len_fits(c, len) || !len_fits(c, int64_t(len) + grow)) {
                atomicOr(&bad, BITNET_CACHE_ERR_LEN);
            } else {
                it.to = s;
                it.pages = pages_of(c, len);
                it.len = len;
                if (grow > 0 && (len & (ps - 1)) != 0) {
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
        if (ONE) {
            own = it;
            own_add = grow;
        } else {
            w.item[i] = it;
        }
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
        const int32_t p = item(i).from;
        if (p < 0) continue;
        atomicAdd(&w.a[p], 1);
        atomicMax(&w.b[p], static_cast<int32_t>(i));
    }
    __syncthreads();
    long long want = 0;  // pages that the call needs
    for (int64_t i = threadIdx.x; i < n; i += kPlanThreads) {
        Item it = item(i);
        if (it.to < 0) continue;
        if (it.from >= 0 && __ldcg(&w.a[it.from]) == c.refs[it.from] &&
            __ldcg(&w.b[it.from]) == i) {
            it.from = -1;  // all holders grow, and this is the last: it keeps the page
            if (ONE)
                own.from = -1;
            else
                w.item[i].from = -1;
        }
        want += pages_of(c, it.len + more(i)) - it.pages + (it.from >= 0);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) want += __shfl_xor_sync(0xFFFFFFFFu, want, d);
    if ((threadIdx.x & 31) == 0) wants[threadIdx.x >> 5] = want;
    __syncthreads();
    int64_t total = wants[threadIdx.x & 31];
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    // The lowest `total` free pages, ascending, into a (the marks in a and b are done with).
    int64_t found = 0;
    for (int64_t base = 0; base < c.num_pages && found < total; base += 32768) {
        const uint32_t word = ~live_word(c, base);
        int all;
        const int64_t rank = found + block_scan(__popc(word), &all);
        for_pages(base, word, rank, total, [&](int64_t r, int32_t p) { w.a[r] = p; });
        found += all;
    }
    __syncthreads();
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
        if (i < n) it = item(i);
        const bool cow = it.to >= 0 && it.from >= 0;
        if (it.to >= 0) {
            grown = pages_of(c, it.len + more(i));
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
            copies[2 + 2 * int64_t(slot)] = it.from;
            copies[3 + 2 * int64_t(slot)] = w.a[rank];
            atomicSub(&c.refs[it.from], 1);
        }
        for (int j = it.pages - cow; j < grown; ++j) {
            const int32_t p = w.a[rank++];
            row[j] = p;
            c.refs[p] = 1;
        }
        c.lens[it.to] = it.len + more(i);
    }
    if (threadIdx.x == 0) {
        copies[0] = copy_base;
        copies[1] = 0;
    }
}

// A table entry after a compaction. The plan leaves a[k], the k-th free page below `live`, and
// for page p from `live` on a[p] = its rank among those in use, or -1.
__device__ __forceinline__ void move_page(const CacheView& c, const Ws& w, int32_t live,
                                          int32_t* entry) {
    const int32_t p = *entry;
    if (uint32_t(p) < uint32_t(live)) return;
    const int32_t rank = uint32_t(p) >= uint32_t(c.num_pages) ? -1 : w.a[p];
    if (rank < 0)
        atomicOr(c.error, BITNET_CACHE_ERR_PAGE);
    else
        *entry = w.a[rank];
}

// The k-th move of a compaction: its pair, and the counts.
__device__ __forceinline__ void move_count(const CacheView& c, const Ws& w, int32_t* copies,
                                           int64_t k) {
    const int32_t from = w.b[k], to = w.a[k];
    *reinterpret_cast<int2*>(copies + 2 + 2 * k) = make_int2(from, to);
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
}

// Pages that slot s holds, 0 (and a report) for a length that does not fit.
__device__ __forceinline__ int32_t slot_pages(const CacheView& c, int64_t s, bool report) {
    const int32_t len = c.lens[s];
    if (len_fits(c, len)) return pages_of(c, len);
    if (report) atomicOr(c.error, BITNET_CACHE_ERR_LEN);
    return 0;
}

// Compact, first step, in one CTA: with L pages in use, lists the used pages from L on (b) and the
// free ones below L (a), both ascending. `alone`: the same CTA does the second step too, a warp per
// slot.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(CacheView c, Ws w,
                                                                    int32_t* copies, int alone) {
    pdl_trigger();
    pdl_wait();
    auto valid_of = [&](int64_t base) {
        const int64_t rest = c.num_pages - (base + 32 * threadIdx.x);
        return rest >= 32 ? ~0u : rest <= 0 ? 0u : (1u << rest) - 1;
    };
    int live = 0;
    uint32_t word = 0;  // of the last 32768 pages: all of them, in most pools
    for (int64_t base = 0; base < c.num_pages; base += 32768) {
        int all;
        word = live_word(c, base) & valid_of(base);
        block_scan(__popc(word), &all);
        live += all;
    }
    int holes = 0, movers = 0;
    for (int64_t base = 0; base < c.num_pages; base += 32768) {
        const int64_t low = int64_t(live) - (base + 32 * threadIdx.x);
        const uint32_t below = low >= 32 ? ~0u : low <= 0 ? 0u : (1u << low) - 1;
        const uint32_t valid = valid_of(base);
        if (c.num_pages > 32768) word = live_word(c, base) & valid;
        const uint32_t hole = ~word & valid & below, mover = word & ~below;
        int all;  // both counts in one scan: at most 32768 each
        const int ranks = block_scan(__popc(hole) | __popc(mover) << 16, &all);
        for_pages(base, hole, holes + (ranks & 0xFFFF), INT32_MAX,
                  [&](int64_t r, int32_t p) { w.a[r] = p; });
        for_pages(base, mover, movers + (uint32_t(ranks) >> 16), INT32_MAX,
                  [&](int64_t r, int32_t p) {
                      w.b[r] = p;
                      w.a[p] = static_cast<int32_t>(r);
                  });
        for_pages(base, ~word & valid & ~below, 0, INT32_MAX,  // nobody may hold these
                  [&](int64_t, int32_t p) { w.a[p] = -1; });
        holes += all & 0xFFFF;
        movers += uint32_t(all) >> 16;
    }
    if (threadIdx.x == 0) {
        copies[0] = movers;
        copies[1] = 0;
        w.head[1] = live;
        w.head[2] = movers;
    }
    if (!alone) return;
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += kPlanThreads) move_count(c, w, copies, k);
    for (int64_t s = threadIdx.x >> 5; s < c.max_seqs; s += kPlanThreads / 32) {
        const int32_t pages = slot_pages(c, s, (threadIdx.x & 31) == 0);
        for (int32_t j = threadIdx.x & 31; j < pages; j += 32)
            move_page(c, w, live, c.table + s * c.max_pages + j);
    }
}

// Compact, second step: the moves over all threads of the grid, then the tables, blockIdx.x walking
// a row in chunks and blockIdx.y the slots.
__global__ void __launch_bounds__(kApplyThreads) compact_apply_kernel(CacheView c, Ws w,
                                                                      int32_t* copies) {
    pdl_trigger();
    pdl_wait();
    const int32_t live = w.head[1], movers = w.head[2];
    const int64_t ctas = int64_t(gridDim.x) * gridDim.y;
    for (int64_t k = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kApplyThreads + threadIdx.x;
         k < movers; k += ctas * kApplyThreads)
        move_count(c, w, copies, k);
    for (int64_t s = blockIdx.y; s < c.max_seqs; s += gridDim.y) {
        const int32_t pages = slot_pages(c, s, threadIdx.x == 0);
        int32_t* row = c.table + s * c.max_pages;
        for (int64_t j0 = int64_t(blockIdx.x) * kApplyChunk; j0 < pages;
             j0 += int64_t(gridDim.x) * kApplyChunk) {
#pragma unroll
            for (int u = 0; u < kApplyChunk / kApplyThreads; ++u) {
                const int64_t j = j0 + u * kApplyThreads + threadIdx.x;
                if (j < pages) move_page(c, w, live, row + j);
            }
        }
    }
}

// Copies pages: the work is cut into pieces of 16 KB (256 threads x 4 x 16 bytes) over all pairs,
// layers and pools, and the grid strides over them. Bound by HBM: every byte read and written once
// (about 4000 pages of 64 KB in two layers at 6.3 TB/s).
constexpr int kCopyPieces = 4;
constexpr int64_t kCopyUnit = int64_t(kApplyThreads) * kCopyPieces * 16;

__global__ void __launch_bounds__(kApplyThreads) copy_kernel(CacheView c,
                                                             const __grid_constant__ CacheLayers l,
                                                             int nlayers, const int32_t* copies,
                                                             int64_t max_copies) {
    pdl_trigger();
    pdl_wait();
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

// Writes new tokens. A CTA takes about 2048 pieces of 8 values (kv_heads * D / 4 pieces a token),
// eight per thread on their way at once (with four 32768 tokens took 52 µs instead of 47), while
// some of its threads look up where the tokens go; D / 8 neighbouring lanes hold a row, so its
// absolute maximum is one warp reduction away. Bound by HBM (K and V read once, pages written
// once: 32768 tokens of 8 heads of 128 in bf16 at 5.7 TB/s), or by latency for one token per
// sequence.
constexpr int kAppendPieces = 8;
constexpr int kAppendTokens = 128;  // tokens of a CTA: 2048 pieces of the smallest

template <int D>
__global__ void __launch_bounds__(kApplyThreads) append_kernel(CacheView c, bitnet_cache_layer lay,
                                                               const uint16_t* k,
                                                               const uint16_t* v, int64_t T,
                                                               int tokens, const int32_t* seqs,
                                                               const int32_t* pos) {
    constexpr int kLanes = D / 8;
    __shared__ int32_t rows[kAppendTokens];  // first row of the token in the pools, or -1
    pdl_trigger();
    pdl_wait();
    const int64_t t0 = int64_t(blockIdx.x) * tokens;
    const int here = static_cast<int>(T - t0 < tokens ? T - t0 : tokens);
    const int half = c.kv_heads * kLanes;  // pieces of a token's K
    const int pieces = here * 2 * half;
    for (int p0 = 0; p0 < pieces; p0 += kAppendPieces * kApplyThreads) {
        uint4 x[kAppendPieces];
        int tok[kAppendPieces], at[kAppendPieces];
#pragma unroll
        for (int u = 0; u < kAppendPieces; ++u) {
            const int p = p0 + u * kApplyThreads + threadIdx.x;
            tok[u] = -1;
            if (p >= pieces) continue;
            tok[u] = p / (2 * half);
            at[u] = p - tok[u] * 2 * half;
            const bool is_v = at[u] >= half;
            x[u] = __ldg(reinterpret_cast<const uint4*>(is_v ? v : k) + (t0 + tok[u]) * half +
                         (is_v ? at[u] - half : at[u]));
        }
        if (p0 == 0) {
            if (threadIdx.x < here) {
                const int64_t t = t0 + threadIdx.x;
                const int64_t s = seqs ? seqs[t] : t;
                int32_t row = -1, err = 0;
                if (s >= c.max_seqs) {
                    err = BITNET_CACHE_ERR_SEQ;
                } else if (s >= 0) {
                    const int32_t len = c.lens[s], j = pos ? pos[t] : len - 1;
                    if (j < 0 || j >= len || !len_fits(c, len)) {
                        err = BITNET_CACHE_ERR_LEN;
                    } else {
                        const int32_t page = c.table[s * c.max_pages + (j >> c.page_shift)];
                        if (uint32_t(page) >= uint32_t(c.num_pages))
                            err = BITNET_CACHE_ERR_PAGE;
                        else
                            row = ((page * c.kv_heads) << c.page_shift) +
                                  (j & ((1 << c.page_shift) - 1));
                    }
                }
                if (err) atomicOr(c.error, err);
                rows[threadIdx.x] = row;
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kAppendPieces; ++u) {
            if (tok[u] < 0 || rows[tok[u]] < 0) continue;  // kLanes neighbours alike
            const bool is_v = at[u] >= half;
            const int in = is_v ? at[u] - half : at[u], head = in / kLanes, piece = in % kLanes;
            const int64_t to = rows[tok[u]] + (head << c.page_shift);
            if (!c.i8) {
                reinterpret_cast<uint4*>(is_v ? lay.v : lay.k)[to * kLanes + piece] = x[u];
                continue;
            }
            // bf16 magnitudes order as unsigned integers, Inf and NaN behind the others: an exact
            // maximum over the row's lanes. A row with either gets NaN as its scale.
            const uint32_t lanes = ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
            const uint32_t top = __reduce_max_sync(lanes, absmax8_bits(x[u]));
            const float amax = top < 0x7F80u ? fmaxf(bf16_lo(top), kActEps)
                                             : __uint_as_float(0x7FC00000u);
            const float scale = __fdiv_rn(127.0f, amax);
            reinterpret_cast<uint2*>(is_v ? lay.v : lay.k)[to * kLanes + piece] =
                quant8(x[u], scale);
            if (piece == 0) (is_v ? lay.v_scale : lay.k_scale)[to] = scale;
        }
    }
}

// Whether one CTA applies a plan itself, in rounds of a warp per row and 32 entries: up to three
// rounds that takes less than a second launch (fork and free of 6 rows of 39 pages 5.5 against 7.9
// µs, of 32 rows of 64 pages 6.1 against 7.8; eight rounds, 64 rows of 100 pages, 11.4 against 7.8).
bool applies_alone(const CacheView& c, int64_t rows) {
    return ((rows + 31) / 32) * ((c.max_pages + 31) / 32) <= 3;
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
    const bool alone = applies_alone(c, n);
    const cudaError_t e =
        launch_pdl(plan_kernel, dim3(1), kPlanThreads, 0, stream, c, w, src, dst, n, int(alone));
    if (e != cudaSuccess || alone) return e;
    return launch_pdl(apply_kernel<true>, apply_grid(c, n), kApplyThreads, 0, stream, c, w, n);
}

cudaError_t launch_cache_free(const CacheView& c, const int32_t* seqs, int64_t n, void* ws,
                              cudaStream_t stream) {
    const Ws w = ws_split(c, ws);
    const bool alone = applies_alone(c, n);
    const cudaError_t e = launch_pdl(plan_kernel, dim3(1), kPlanThreads, 0, stream, c, w,
                                     static_cast<const int32_t*>(nullptr), seqs, n, int(alone));
    if (e != cudaSuccess || alone) return e;
    return launch_pdl(apply_kernel<false>, apply_grid(c, n), kApplyThreads, 0, stream, c, w, n);
}

cudaError_t launch_cache_extend(const CacheView& c, const int32_t* seqs, const int32_t* add,
                                int64_t n, int32_t* copies, void* ws, cudaStream_t stream) {
    const Ws w = ws_split(c, ws);
    return launch_pdl(n <= kPlanThreads ? extend_kernel<true> : extend_kernel<false>, dim3(1),
                      kPlanThreads, 0, stream, c, w, seqs, add, n, copies);
}

cudaError_t launch_cache_compact(const CacheView& c, int32_t* copies, void* ws,
                                 cudaStream_t stream) {
    const Ws w = ws_split(c, ws);
    const bool alone = applies_alone(c, c.max_seqs);
    const cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), kPlanThreads, 0, stream, c, w,
                                     copies, int(alone));
    if (e != cudaSuccess || alone) return e;
    return launch_pdl(compact_apply_kernel, apply_grid(c, c.max_seqs), kApplyThreads, 0, stream, c,
                      w, copies);
}

cudaError_t launch_cache_copy(const CacheView& c, const CacheLayers& layers, int nlayers,
                              const int32_t* copies, int64_t max_copies, cudaStream_t stream) {
    // Eight CTAs an SM, or fewer where the list cannot hold work for them.
    const int64_t tokens = int64_t(c.kv_heads) << c.page_shift;
    const int64_t units = 2 * nlayers * max_copies *
                          ((tokens * c.head_dim * (c.i8 ? 1 : 2) + kCopyUnit - 1) / kCopyUnit +
                           (c.i8 ? (tokens * 4 + kCopyUnit - 1) / kCopyUnit : 0));
    const int64_t most = int64_t(tc_num_sms()) * 8;
    return launch_pdl(copy_kernel, dim3(static_cast<unsigned>(units < most ? units : most)),
                      kApplyThreads, 0, stream, c, layers, nlayers, copies, max_copies);
}

cudaError_t launch_cache_append(const CacheView& c, const bitnet_cache_layer& layer,
                                const uint16_t* k, const uint16_t* v, int64_t T,
                                const int32_t* seqs, const int32_t* pos, cudaStream_t stream) {
    const int per = c.kv_heads * (c.head_dim / 4);  // pieces of a token
    // as many as eight pieces per thread make, but no fewer CTAs than SMs while there are tokens
    const int full = per >= kAppendPieces * kApplyThreads ? 1 : kAppendPieces * kApplyThreads / per;
    const int64_t even = (T + tc_num_sms() - 1) / tc_num_sms();
    const int tokens = even < full ? static_cast<int>(even) : full;
    const int64_t blocks = (T + tokens - 1) / tokens;
    return launch_pdl(c.head_dim == 64 ? append_kernel<64> : append_kernel<128>,
                      dim3(static_cast<unsigned>(blocks)), kApplyThreads, 0, stream, c, layer, k, v,
                      T, tokens, seqs, pos);
}

}  // namespace bitnet
