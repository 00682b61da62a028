// C-ABI host layer of the decode-step operators: argument checks and launches of the 4-bit
// linear layers, the paged cache's upkeep and the attention over it. Contracts: include/bitnet.h.
#include <cuda_runtime.h>

#include "bitnet.h"
#include "bitnet_internal.h"
#include "cache_internal.h"

namespace bitnet {
namespace {

bitnet_status check_cache(const bitnet_cache* c, CacheView* v) {
    if (!c || !c->table || !c->lens || !c->refs || !c->error) return BITNET_ERR_NULL;
    if (c->num_pages < 1 || c->num_pages > (int64_t(1) << 30) || c->max_seqs < 1 ||
        c->max_seqs > (int64_t(1) << 24) || c->kv_heads < 1 || c->kv_heads > 1024)
        return BITNET_ERR_SHAPE;
    int shift = 3;
    while (shift <= 8 && (1 << shift) != c->page_size) ++shift;
    if (shift > 8) return BITNET_ERR_UNSUPPORTED;
    // (positions, rounded up to a kernel's step, stay in 32 bits)
    if (c->max_pages < 1 || c->max_pages > (int64_t(1) << (30 - shift))) return BITNET_ERR_SHAPE;
    // Rows of a pool are numbered in 32 bits (2^31 of the smallest would be 137 GB of K alone).
    if ((c->num_pages * c->kv_heads) << shift >= (int64_t(1) << 31)) return BITNET_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return BITNET_ERR_UNSUPPORTED;
    if (c->dtype != BITNET_CACHE_BF16 && c->dtype != BITNET_CACHE_I8) return BITNET_ERR_UNSUPPORTED;
    if (!aligned(c->table, 4) || !aligned(c->lens, 4) || !aligned(c->refs, 4) ||
        !aligned(c->error, 4))
        return BITNET_ERR_ALIGN;
    *v = CacheView{c->table,
                   c->lens,
                   c->refs,
                   c->error,
                   c->max_pages,
                   static_cast<int32_t>(c->num_pages),
                   static_cast<int32_t>(c->max_seqs),
                   c->kv_heads,
                   shift,
                   c->head_dim,
                   c->dtype == BITNET_CACHE_I8};
    return BITNET_OK;
}

bitnet_status check_layer(const CacheView& c, const bitnet_cache_layer& l) {
    if (!l.k || !l.v || (c.i8 && (!l.k_scale || !l.v_scale))) return BITNET_ERR_NULL;
    if (!aligned(l.k, 16) || !aligned(l.v, 16) ||
        (c.i8 && (!aligned(l.k_scale, 16) || !aligned(l.v_scale, 16))))
        return BITNET_ERR_ALIGN;
    return BITNET_OK;
}

// Lists hold up to 2^24 entries, as many as there can be slots.
bitnet_status check_list(int64_t n) {
    return (n < 1 || n > (int64_t(1) << 24)) ? BITNET_ERR_SHAPE : BITNET_OK;
}

bitnet_status check_ws(const void* ws, size_t bytes, size_t need) {
    if (!ws || bytes < need) return BITNET_ERR_WORKSPACE;
    return aligned(ws, 256) ? BITNET_OK : BITNET_ERR_ALIGN;
}

size_t upkeep_ws(const CacheView& c, int64_t n) {
    return cache_ws_bytes(c.num_pages, c.max_seqs, n);
}

// Queries and heads of an attention call.
bitnet_status check_heads(int32_t kv_heads, int64_t B, int64_t heads) {
    if (B < 1 || B > (int64_t(1) << 20) || heads < 1 || heads > 16384 || heads % kv_heads != 0)
        return BITNET_ERR_SHAPE;
    return BITNET_OK;
}

}  // namespace
}  // namespace bitnet

using namespace bitnet;

extern "C" {

int64_t bitnet_w4_row_bytes(int64_t K) { return K < 1 ? 0 : w4_row_bytes(K); }

bitnet_status bitnet_pack_w4(const float* W, int64_t N, int64_t K, int32_t group, uint8_t* packed,
                             uint16_t* scales, void* stream) {
    if (!W || !packed || !scales) return BITNET_ERR_NULL;
    bitnet_status st = check_mk(1, K);
    if (st != BITNET_OK) return st;
    if ((st = check_n(N)) != BITNET_OK) return st;
    if (group != 32 && group != 64 && group != 128) return BITNET_ERR_UNSUPPORTED;
    if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(scales, 2)) return BITNET_ERR_ALIGN;
    return from_cuda(
        launch_pack_w4(W, N, K, group, packed, scales, static_cast<cudaStream_t>(stream)));
}

bitnet_status bitnet_linear_w4(const uint16_t* x, int64_t M, int64_t K, const uint8_t* packed,
                               const uint16_t* scales, int32_t group, int64_t N, void* y,
                               bitnet_out_dtype out_dtype, void* stream) {
    if (!x || !packed || !scales || !y) return BITNET_ERR_NULL;
    bitnet_status st = check_mk(M, K);
    if (st != BITNET_OK) return st;
    if ((st = check_n(N)) != BITNET_OK) return st;
    if (group != 32 && group != 64 && group != 128) return BITNET_ERR_UNSUPPORTED;
    if (out_dtype != BITNET_OUT_BF16 && out_dtype != BITNET_OUT_F32) return BITNET_ERR_UNSUPPORTED;
    if (K > int64_t(group) * BITNET_W4_MAX_GROUPS) return BITNET_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scales, 2) || !aligned(y, 16))
        return BITNET_ERR_ALIGN;
    return from_cuda(launch_linear_w4(x, M, K, packed, scales, group, N, y,
                                      out_dtype == BITNET_OUT_F32,
                                      static_cast<cudaStream_t>(stream)));
}

size_t bitnet_cache_workspace_size(const bitnet_cache* cache, int64_t n) {
    CacheView c;
    if (check_cache(cache, &c) != BITNET_OK || n < 0 || n > (int64_t(1) << 24)) return 0;
    return upkeep_ws(c, n);
}

bitnet_status bitnet_cache_fork(const bitnet_cache* cache, const int32_t* src, const int32_t* dst,
                                int64_t n, void* workspace, size_t workspace_bytes, void* stream) {
    CacheView c;
    bitnet_status st = check_cache(cache, &c);
    if (st != BITNET_OK) return st;
    if (!src || !dst) return BITNET_ERR_NULL;
    if ((st = check_list(n)) != BITNET_OK) return st;
    if (!aligned(src, 4) || !aligned(dst, 4)) return BITNET_ERR_ALIGN;
    if ((st = check_ws(workspace, workspace_bytes, upkeep_ws(c, n))) != BITNET_OK) return st;
    return from_cuda(
        launch_cache_fork(c, src, dst, n, workspace, static_cast<cudaStream_t>(stream)));
}

bitnet_status bitnet_cache_extend(const bitnet_cache* cache, const int32_t* seqs,
                                  const int32_t* add, int64_t n, int32_t* copies,
                                  int64_t max_copies, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    CacheView c;
    bitnet_status st = check_cache(cache, &c);
    if (st != BITNET_OK) return st;
    if (!seqs || !add || !copies) return BITNET_ERR_NULL;
    if ((st = check_list(n)) != BITNET_OK) return st;
    if (!aligned(seqs, 4) || !aligned(add, 4) || !aligned(copies, 8)) return BITNET_ERR_ALIGN;
    if (max_copies < n) return BITNET_ERR_WORKSPACE;
    if ((st = check_ws(workspace, workspace_bytes, upkeep_ws(c, n))) != BITNET_OK) return st;
    return from_cuda(launch_cache_extend(c, seqs, add, n, copies, workspace,
                                         static_cast<cudaStream_t>(stream)));
}

bitnet_status bitnet_cache_free(const bitnet_cache* cache, const int32_t* seqs, int64_t n,
                                void* workspace, size_t workspace_bytes, void* stream) {
    CacheView c;
    bitnet_status st = check_cache(cache, &c);
    if (st != BITNET_OK) return st;
    if (!seqs) return BITNET_ERR_NULL;
    if ((st = check_list(n)) != BITNET_OK) return st;
    if (!aligned(seqs, 4)) return BITNET_ERR_ALIGN;
    if ((st = check_ws(workspace, workspace_bytes, upkeep_ws(c, n))) != BITNET_OK) return st;
    return from_cuda(launch_cache_free(c, seqs, n, workspace, static_cast<cudaStream_t>(stream)));
}

bitnet_status bitnet_cache_compact(const bitnet_cache* cache, int32_t* copies, int64_t max_copies,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    CacheView c;
    bitnet_status st = check_cache(cache, &c);
    if (st != BITNET_OK) return st;
    if (!copies) return BITNET_ERR_NULL;
    if (!aligned(copies, 8)) return BITNET_ERR_ALIGN;
    if (max_copies < c.num_pages / 2) return BITNET_ERR_WORKSPACE;
    if ((st = check_ws(workspace, workspace_bytes, upkeep_ws(c, 0))) != BITNET_OK) return st;
    return from_cuda(
        launch_cache_compact(c, copies, workspace, static_cast<cudaStream_t>(stream)));
}

bitnet_status bitnet_cache_copy(const bitnet_cache* cache, const bitnet_cache_layer* layers,
                                int32_t nlayers, const int32_t* copies, int64_t max_copies,
                                void* stream) {
    CacheView c;
    bitnet_status st = check_cache(cache, &c);
    if (st != BITNET_OK) return st;
    if (!layers || !copies) return BITNET_ERR_NULL;
    if (nlayers < 1 || nlayers > BITNET_CACHE_MAX_LAYERS || max_copies < 0 ||
        max_copies > (int64_t(1) << 30))
        return BITNET_ERR_SHAPE;
    if (!aligned(copies, 8)) return BITNET_ERR_ALIGN;
    CacheLayers l = {};
    for (int i = 0; i < nlayers; ++i) {
        if ((st = check_layer(c, layers[i])) != BITNET_OK) return st;
        l.layer[i] = layers[i];
    }
    if (max_copies == 0) return BITNET_OK;
    return from_cuda(launch_cache_copy(c, l, nlayers, copies, max_copies,
                                       static_cast<cudaStream_t>(stream)));
}

bitnet_status bitnet_cache_append(const bitnet_cache* cache, const bitnet_cache_layer* layer,
                                  const uint16_t* k, const uint16_t* v, int64_t T,
                                  const int32_t* seqs, const int32_t* pos, void* stream) {
    CacheView c;
    bitnet_status st = check_cache(cache, &c);
    if (st != BITNET_OK) return st;
    if (!layer || !k || !v) return BITNET_ERR_NULL;
    if (T < 1 || T >= (int64_t(1) << 31)) return BITNET_ERR_SHAPE;
    if ((st = check_layer(c, *layer)) != BITNET_OK) return st;
    if (!aligned(k, 16) || !aligned(v, 16) || (seqs && !aligned(seqs, 4)) ||
        (pos && !aligned(pos, 4)))
        return BITNET_ERR_ALIGN;
    return from_cuda(launch_cache_append(c, *layer, k, v, T, seqs, pos,
                                         static_cast<cudaStream_t>(stream)));
}

size_t bitnet_paged_attention_workspace_size(const bitnet_cache* cache, int64_t B, int64_t heads) {
    CacheView c;
    if (check_cache(cache, &c) != BITNET_OK || check_heads(c.kv_heads, B, heads) != BITNET_OK)
        return 0;
    return attn_ws_bytes(c.head_dim);
}

bitnet_status bitnet_paged_attention(const bitnet_cache* cache, const bitnet_cache_layer* layer,
                                     const uint16_t* q, int64_t B, int64_t heads,
                                     const int32_t* seqs, float scale, int64_t window,
                                     int64_t sinks, uint16_t* out, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    AttnParams p;
    bitnet_status st = check_cache(cache, &p.c);
    if (st != BITNET_OK) return st;
    if (!layer || !q || !out) return BITNET_ERR_NULL;
    if ((st = check_heads(p.c.kv_heads, B, heads)) != BITNET_OK) return st;
    if (window < 0 || sinks < 0) return BITNET_ERR_SHAPE;
    // (times log2 e it stays finite)
    if (!(scale > -2.0e38f && scale < 2.0e38f)) return BITNET_ERR_UNSUPPORTED;
    if ((st = check_layer(p.c, *layer)) != BITNET_OK) return st;
    if (!aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4)) ||
        (seqs && !aligned(seqs, 4)))
        return BITNET_ERR_ALIGN;
    if ((st = check_ws(workspace, workspace_bytes, attn_ws_bytes(p.c.head_dim))) != BITNET_OK)
        return st;
    // Lengths are at most 2^30, so a window or sinks beyond that see everything they can.
    const int64_t cap = (int64_t(1) << 31) - 1;
    p.layer = *layer;
    p.q = q;
    p.seqs = seqs;
    p.out = out;
    p.lse = lse;
    p.ws = workspace;
    p.scale = scale;
    p.B = static_cast<int32_t>(B);
    p.heads = static_cast<int32_t>(heads);
    p.window = static_cast<int32_t>(window < cap ? window : cap);
    p.sinks = static_cast<int32_t>(sinks < cap ? sinks : cap);
    return from_cuda(launch_paged_attention(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
