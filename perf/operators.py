"""Measured cases of the operators that a decode step needs beside the ternary projections:
matrix-vector products with 4-bit weights and group scales, attention of one new token over a
paged key/value cache, the write of new tokens into that cache, and the upkeep of its pages
(fork, extend with copy on write, free, compact, copy).

`run` computes each one in its plain form (elementary torch operations, 32 bits) while `own` is
False, and through the framework's calls while it is True. `exact` gives the same outputs from
the definitions in 64 bits. Layouts and definitions:

4-bit weights. t[n, k] in [-8, 7], stored as code t + 8. A row is cut into blocks of 128 weights
(the last one filled up with code 8) of 64 bytes, i.e. 16 little-endian 32-bit words; word
4c + j holds weights 32j + 8c .. 32j + 8c + 7 of the block, the even ones in nibbles 0..3 and
the odd ones in nibbles 4..7. Scales are bf16, (N, ceil(K / group)).
    y[m, n] = sum_g scale[n, g] * sum_{k in g} x[m, k] * t[n, k]

Cache. Pools of pages (num_pages, kv_heads, page_size, head_dim) for K and for V in bf16, or in
int8 with one fp32 scale per token and head, (num_pages, kv_heads, page_size), value = q / scale.
Sequence slot s holds lens[s] tokens, token j in page table[s, j // page_size]; refs[p] counts
the holders of page p, and a page is free while it is 0.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the benchmark's smallest projection (640 x 2560) kept in 4 bits, one token: latency
        dict(name="w4_kv_m1", kind="w4", M=1, N=640, K=2560, group=128, out="bf16"),
        # an MLP's down projection (2560 x 6912), the layer mixed-precision setups keep wider
        dict(name="w4_down_m1", kind="w4", M=1, N=2560, K=6912, group=64, out="bf16"),
        # a 14336 x 4096 MLP projection for a batch of eight sequences
        dict(name="w4_mlp_m8", kind="w4", M=8, N=14336, K=4096, group=128, out="bf16"),
        # logits over a large vocabulary of odd size, a few tokens, fp32 out, finest groups
        dict(name="w4_logits_m3", kind="w4", M=3, N=131071, K=4096, group=32, out="f32"),
        # one sequence of 4096 tokens, 20 heads over 5 key/value heads: latency
        dict(name="attn_one", kind="attn", B=1, heads=20, kv=5, D=128, page=16, low=4096,
             high=4096, dtype="bf16", window=0, sinks=0),
        # a ragged serving batch, empty and single-token rows among them
        dict(name="attn_ragged", kind="attn", B=48, heads=32, kv=8, D=128, page=64, low=0,
             high=8192, dtype="bf16", window=0, sinks=0),
        # few long sequences over an 8-bit cache
        dict(name="attn_long_i8", kind="attn", B=8, heads=32, kv=8, D=128, page=128, low=4097,
             high=65536, dtype="i8", window=0, sinks=0),
        # a sliding window with four sinks over long caches, small heads
        dict(name="attn_window", kind="attn", B=64, heads=32, kv=8, D=64, page=32, low=100,
             high=24576, dtype="bf16", window=4096, sinks=4),
        # one new token for each of 64 sequences, quantised into an 8-bit cache: latency
        dict(name="append_step_i8", kind="append", T=64, seqs=64, kv=5, D=128, page=16,
             dtype="i8"),
        # prompts of several sequences written at once
        dict(name="append_prompt", kind="append", T=32768, seqs=7, kv=8, D=128, page=64,
             dtype="bf16"),
        # beams forked from two sequences in a small cache: latency of the bookkeeping
        dict(name="pages_small", kind="pages", parents=2, fan=3, pages=256, page=16, kv=5, D=128,
             layers=2, low=100, high=600, dtype="bf16"),
        # upkeep of a large, scattered cache: most of the time is moving pages
        dict(name="pages_large", kind="pages", parents=32, fan=7, pages=16384, page=16, kv=8,
             D=128, layers=2, low=1000, high=6000, dtype="bf16"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["w4", "attn", "append", "pages"])
    if kind == "w4":
        while True:
            c = dict(kind=kind, M=rng.choice([1, 1, 2, 3, 5, 8, 16]), N=_log_int(rng, 33, 131071),
                     K=64 * _log_int(rng, 4, 224), group=rng.choice([32, 64, 128]),
                     out=rng.choice(["bf16", "f32"]))
            if c["N"] * c["K"] <= 131071 * 4096:
                return c
    if kind == "attn":
        while True:
            kv = rng.choice([1, 2, 5, 8])
            c = dict(kind=kind, B=_log_int(rng, 1, 128), heads=kv * rng.choice([1, 3, 4, 8]),
                     kv=kv, D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                     low=0, high=_log_int(rng, 16, 65536), dtype=rng.choice(["bf16", "i8"]),
                     window=0, sinks=0)
            c["low"] = rng.choice([0, 1, c["high"] // 2, c["high"]])
            if rng.random() < 0.4:
                c["window"] = _log_int(rng, 1, 8192)
                c["sinks"] = rng.choice([0, 1, 4, 37])
            if c["B"] * c["high"] * kv * c["D"] <= 48 * 8192 * 8 * 128:
                return c
    if kind == "append":
        seqs = _log_int(rng, 1, 128)
        return dict(kind=kind, T=max(seqs, _log_int(rng, 1, 32768)), seqs=seqs,
                    kv=rng.choice([1, 2, 5, 8]), D=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "i8"]))
    while True:
        c = dict(kind=kind, parents=_log_int(rng, 1, 32), fan=rng.randint(1, 7),
                 pages=_log_int(rng, 128, 16384), page=rng.choice([16, 32, 64]),
                 kv=rng.choice([1, 2, 5, 8]), D=rng.choice([64, 128]), layers=rng.randint(1, 3),
                 low=1, high=_log_int(rng, 50, 6000), dtype=rng.choice(["bf16", "i8"]))
        held = c["parents"] * -(-c["high"] // c["page"])
        size = c["pages"] * c["page"] * c["kv"] * c["D"] * c["layers"]
        if held + 2 * c["parents"] * (c["fan"] + 1) <= c["pages"] and \
                size <= 16384 * 16 * 8 * 128 * 2:
            return c


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _pack_w4(t):
    """Codes t (N, K) int8 in [-8, 7] -> (N, 64 ceil(K / 128)) uint8 in the layout above."""
    N, K = t.shape
    pad = -K % 128
    c = torch.nn.functional.pad(t, (0, pad)).add_(8).to(torch.uint8)
    c = c.view(N, (K + pad) // 128, 4, 4, 8).transpose(2, 3)
    c = torch.cat([c[..., 0::2], c[..., 1::2]], dim=-1)
    return (c[..., 0::2] | c[..., 1::2] << 4).reshape(N, (K + pad) // 2).contiguous()


def _unpack_w4(packed, K):
    """The inverse of _pack_w4, as int8 values t (N, K)."""
    N = packed.shape[0]
    b = packed.view(N, -1, 4, 4, 4)
    c = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)
    c = torch.stack([c[..., :4], c[..., 4:]], dim=-1).flatten(-2)
    return c.transpose(2, 3).reshape(N, -1)[:, :K].to(torch.int8) - 8


def _quantise(x):
    """One scale per last axis: s = 127 / max(max |x|, 1e-5), q = rint(x s), as the framework's
    activation quantiser."""
    amax = x.float().abs().amax(-1).clamp(min=1e-5)
    s = torch.full_like(amax, 127.0) / amax  # one division (127.0 / amax would be two steps)
    return torch.round(x.float() * s[..., None]).to(torch.int8), s


def _pools(g, c, pages, layers):
    shape = (pages, c["kv"], c["page"], c["D"])
    made = []
    for _ in range(layers):
        layer = {}
        for w in ("k", "v"):
            if c["dtype"] == "i8":
                layer[w], layer[w + "_scale"] = _quantise(_randn(g, *shape))
            else:
                layer[w], layer[w + "_scale"] = _randn(g, *shape), None
        made.append(layer)
    return made


def _lengths(g, n, low, high):
    if high <= low:
        return torch.full((n,), high, dtype=torch.int64)
    lens = torch.randint(low, high + 1, (n,), generator=g, device=DEV)
    lens[0] = high
    if n > 1:
        lens[n - 1] = low
    if n > 2 and low <= 1:
        lens[n // 2] = 1
    return lens.cpu()


def _meta(slots, width, pages):
    """Table, lengths and reference counts as views of one int32 buffer."""
    flat = torch.zeros(slots * width + slots + pages, dtype=torch.int32, device=DEV)
    return flat, dict(table=flat[:slots * width].view(slots, width),
                      lens=flat[slots * width:slots * width + slots],
                      refs=flat[slots * width + slots:])


def _place(g, meta, lens, page, pages):
    """Gives every sequence its pages, scattered over the pool."""
    need = -(-lens // page)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    ends = torch.cumsum(need, 0)
    meta["table"].fill_(-1)
    for s, (n, e) in enumerate(zip(need.tolist(), ends.tolist())):
        meta["table"][s, :n] = perm[e - n:e]
    meta["refs"].zero_()
    meta["refs"][perm[:int(ends[-1])].long()] = 1
    meta["lens"].zero_()
    meta["lens"][:len(lens)] = lens.to(DEV, torch.int32)


def _cache(c, meta, layers):
    """The framework's handle of the cache: pointers and sizes of the tensors above."""
    import ternary_w2a8_linear_token_b200 as bn
    return bn.PagedCache(meta["table"], meta["lens"], meta["refs"], [tuple(
        layer[w] for w in ("k", "v", "k_scale", "v_scale")) for layer in layers])


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["kind"] == "w4":
        t = torch.randn(c["N"], c["K"], generator=g, device=DEV).mul_(2.5).round_()
        t = t.clamp_(-8, 7).to(torch.int8)
        groups = -(-c["K"] // c["group"])
        scales = torch.rand(c["N"], groups, generator=g, device=DEV) * 0.01 + 0.005
        return dict(case=c, x=_randn(g, c["M"], c["K"]), packed=_pack_w4(t),
                    scales=scales.to(torch.bfloat16))
    if c["kind"] == "attn":
        lens = _lengths(g, c["B"], c["low"], c["high"])
        need = int((-(-lens // c["page"])).sum())
        width = max(1, -(-c["high"] // c["page"]))
        _, meta = _meta(c["B"], width, need + 1)
        _place(g, meta, lens, c["page"], need + 1)
        st = dict(case=c, q=_randn(g, c["B"], c["heads"], c["D"]), meta=meta,
                  layers=_pools(g, c, need + 1, 1), high=c["high"])
    elif c["kind"] == "append":
        # each sequence brings T / seqs new tokens behind a few that it holds already
        held = torch.randint(0, 40, (c["seqs"],), generator=g, device=DEV).cpu()
        new = torch.full((c["seqs"],), c["T"] // c["seqs"], dtype=torch.int64)
        new[:c["T"] % c["seqs"]] += 1
        lens = held + new
        width = -(-(40 + -(-c["T"] // c["seqs"])) // c["page"])
        need = c["seqs"] * width
        _, meta = _meta(c["seqs"], width, need)
        _place(g, meta, lens, c["page"], need)
        seqs = torch.repeat_interleave(torch.arange(c["seqs"]), new)
        first = torch.cumsum(new, 0) - new
        pos = torch.arange(c["T"]) - first[seqs] + held[seqs]
        st = dict(case=c, meta=meta, layers=_pools(g, c, need, 1),
                  k=_randn(g, c["T"], c["kv"], c["D"]), v=_randn(g, c["T"], c["kv"], c["D"]),
                  seqs=seqs.to(DEV, torch.int32), pos=pos.to(DEV, torch.int32))
    else:
        # parents hold pages scattered over the pool; the children's slots are empty
        P, kids = c["parents"], c["parents"] * c["fan"]
        lens = _lengths(g, P, c["low"], c["high"])
        flat, meta = _meta(P + kids, -(-c["high"] // c["page"]) + 1, c["pages"])
        _place(g, meta, lens, c["page"], c["pages"])
        work, meta = flat.clone(), meta
        slots = torch.arange(P + kids, device=DEV, dtype=torch.int32)
        dropped = slots[P:][torch.randperm(kids, generator=g, device=DEV)[:(kids + 1) // 2]]
        st = dict(case=c, start=work, flat=flat, meta=meta,
                  layers=_pools(g, c, c["pages"], c["layers"]),
                  src=(torch.arange(kids, device=DEV) % P).to(torch.int32), dst=slots[P:],
                  seqs=slots, dropped=dropped.contiguous(),
                  add=torch.randint(1, c["page"] + 1, (P + kids,), generator=g,
                                    device=DEV).to(torch.int32))
    st["cache"] = _cache(c, st["meta"], st["layers"]) if own else None
    return st


# --------------------------------------------------------------------------- one pass
def run(state):
    kind = state["case"]["kind"]
    if kind == "w4":
        return _run_w4(state)
    if kind == "attn":
        return _run_attn(state)
    if kind == "append":
        return _run_append(state)
    return _run_pages(state)


def _run_w4(st):
    c = st["case"]
    dtype = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    if own:
        import ternary_w2a8_linear_token_b200 as bn
        return bn.bitnet_linear_w4(st["x"], st["packed"], st["scales"], c["group"],
                                   out_dtype=dtype)
    t = _unpack_w4(st["packed"], c["K"])
    s = st["scales"].float().repeat_interleave(c["group"], 1)[:, :c["K"]]
    return (st["x"].float() @ (t.float() * s).T).to(dtype)


def _values(pool, scale):
    return pool.float() if scale is None else pool.float() / scale[..., None]


def _visible(c, lens, width):
    """Positions that a sequence of each length sees, (B, width), and which of them exist:
    all, or the first `sinks` and the last `window` tokens."""
    v = torch.arange(width, device=DEV)
    seen = lens.clamp(max=c["window"] + c["sinks"]) if c["window"] else lens
    skipped = (lens - seen)[:, None]
    return torch.where(v < c["sinks"], v, v + skipped), v < seen[:, None]


def _run_attn(st):
    c = st["case"]
    if own:
        import ternary_w2a8_linear_token_b200 as bn
        out, lse = bn.bitnet_paged_attention(st["q"], st["cache"], 0, window=c["window"],
                                             sinks=c["sinks"], return_lse=True)
        return {"out": out, "lse": lse}
    B, H, KV, D = c["B"], c["heads"], c["kv"], c["D"]
    meta, layer = st["meta"], st["layers"][0]
    width = min(st["high"], c["window"] + c["sinks"]) if c["window"] else st["high"]
    at, there = _visible(c, meta["lens"].long(), max(width, 1))
    at = torch.where(there, at, 0)
    page = torch.gather(meta["table"].long(), 1, at // c["page"]).clamp(min=0)
    off = at % c["page"]
    k = _values(layer["k"][page, :, off],
                None if layer["k_scale"] is None else layer["k_scale"][page, :, off])
    q = st["q"].float().view(B, KV, H // KV, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    del k
    s = s.masked_fill(~there[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    v = _values(layer["v"][page, :, off],
                None if layer["v_scale"] is None else layer["v_scale"][page, :, off])
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return {"out": o.view(B, H, D).to(torch.bfloat16), "lse": lse.view(B, H)}


def _held(layer):
    """What a layer's pages hold: bf16 as it stands, 8 bits as the values they stand for."""
    if layer["k_scale"] is None:
        return [layer["k"], layer["v"]]
    return [_values(layer[w], layer[w + "_scale"]) for w in ("k", "v")]


def _run_append(st):
    c, layer = st["case"], st["layers"][0]
    if own:
        import ternary_w2a8_linear_token_b200 as bn
        bn.bitnet_cache_append(st["cache"], 0, st["k"], st["v"], seqs=st["seqs"], pos=st["pos"])
        return _held(layer)
    page = st["meta"]["table"][st["seqs"].long(), (st["pos"] // c["page"]).long()].long()
    off = (st["pos"] % c["page"]).long()
    for w in ("k", "v"):
        if c["dtype"] == "i8":
            layer[w][page, :, off], layer[w + "_scale"][page, :, off] = _quantise(st[w])
        else:
            layer[w][page, :, off] = st[w]
    return _held(layer)


def _run_pages(st):
    """Children fork from their parents, every sequence grows (shared last pages are copied
    first), half of the children are dropped, and the pool is compacted."""
    c, meta = st["case"], st["meta"]
    st["flat"].copy_(st["start"])  # every pass starts from the same tables
    if own:
        import ternary_w2a8_linear_token_b200 as bn
        cache = st["cache"]
        bn.bitnet_cache_fork(cache, st["src"], st["dst"])
        copies = bn.bitnet_cache_extend(cache, st["seqs"], st["add"])
        bn.bitnet_cache_copy(cache, copies)
        bn.bitnet_cache_free(cache, st["dropped"])
        moves = bn.bitnet_cache_compact(cache)
        bn.bitnet_cache_copy(cache, moves)
        counts = [copies[0], moves[0]]
    else:
        _fork(c, meta, st["src"].long(), st["dst"].long())
        old, new = _extend(c, meta, st["seqs"].long(), st["add"].long())
        _copy(st["layers"], old, new)
        _free(c, meta, st["dropped"].long())
        old2, new2 = _compact(c, meta)
        _copy(st["layers"], old2, new2)
        counts = [torch.tensor(v.numel(), dtype=torch.int32, device=DEV) for v in (old, old2)]
    return {"tables": st["flat"], "counts": counts,
            "pools": [x for layer in st["layers"] for x in _held(layer)]}


def _used(c, meta):
    """Which entries of the table hold pages."""
    col = torch.arange(meta["table"].shape[1], device=DEV)
    return col < ((meta["lens"].long() + c["page"] - 1) // c["page"])[:, None]


def _fork(c, meta, src, dst):
    used = _used(c, meta)[src]
    rows = meta["table"][src]
    meta["table"][dst] = torch.where(used, rows, meta["table"][dst])
    meta["lens"][dst] = meta["lens"][src]
    meta["refs"].index_add_(0, rows.clamp(min=0).flatten().long(),
                            used.flatten().to(torch.int32))


def _extend(c, meta, seqs, add):
    ps, refs = c["page"], meta["refs"]
    lens = meta["lens"][seqs].long()
    had, has = (lens + ps - 1) // ps, (lens + add + ps - 1) // ps
    last = meta["table"][seqs, (had - 1).clamp(min=0)].long().clamp(min=0)
    # a partly filled last page that others hold too is copied before it is written; where all
    # its holders grow in this call, the last of them keeps it
    part = (add > 0) & (lens % ps > 0) & (refs[last] > 1)
    item = torch.arange(len(seqs), device=DEV)
    here = torch.zeros_like(refs, dtype=torch.int64).index_add_(0, last, part.long())
    final = torch.full_like(here, -1).scatter_reduce(0, last, torch.where(part, item, -1),
                                                     "amax")
    keeps = part & (here[last] == refs[last]) & (final[last] == item)
    cow = part & ~keeps
    need = has - had + cow.long()
    begin = torch.cumsum(need, 0) - need
    free = torch.sort((refs > 0).to(torch.int32), stable=True)[1].to(torch.int32)
    col = torch.arange(meta["table"].shape[1], device=DEV)
    fresh = (col >= (had - cow.long())[:, None]) & (col < has[:, None])
    rank = (begin[:, None] + col - (had - cow.long())[:, None]).clamp(0, len(free) - 1)
    meta["table"][seqs] = torch.where(fresh, free[rank], meta["table"][seqs])
    refs.index_add_(0, last, -cow.to(torch.int32))
    refs.index_add_(0, free[rank].flatten().long(), fresh.flatten().to(torch.int32))
    meta["lens"][seqs] = (lens + add).to(torch.int32)
    return last[cow], free[begin[cow]].long()


def _free(c, meta, seqs):
    used = _used(c, meta)[seqs]
    rows = meta["table"][seqs]
    meta["refs"].index_add_(0, rows.clamp(min=0).flatten().long(),
                            -used.flatten().to(torch.int32))
    meta["lens"][seqs] = 0


def _compact(c, meta):
    refs = meta["refs"]
    live = refs > 0
    place = torch.arange(len(refs), device=DEV)
    n = live.sum()
    old = torch.nonzero(live & (place >= n)).flatten()
    new = torch.nonzero(~live & (place < n)).flatten()
    to = place.to(torch.int32)
    to[old] = new.to(torch.int32)
    refs[new] = refs[old]
    refs[old] = 0
    used = _used(c, meta)
    table = meta["table"]
    table.copy_(torch.where(used, to[table.clamp(min=0).long()], table))
    return old, new


def _copy(layers, old, new):
    for layer in layers:
        for x in layer.values():
            if x is not None:
                x[new] = x[old]


# --------------------------------------------------------------------------- what a pass needs
def work(case):
    c = case
    if c["kind"] == "w4":
        groups = -(-c["K"] // c["group"])
        out = 2 if c["out"] == "bf16" else 4
        return {"bytes": c["N"] * c["K"] / 2 + 2 * c["N"] * groups + 2 * c["M"] * c["K"]
                + out * c["M"] * c["N"], "flops": 2 * c["M"] * c["N"] * c["K"]}
    token = 2 * c["kv"] * (c["D"] * 2 if c["dtype"] == "bf16" else c["D"] + 4)
    if c["kind"] == "attn":
        span = c["window"] + c["sinks"] if c["window"] else c["high"]
        low, high = c["low"], c["high"]
        # mean of min(length, span) over lengths spread evenly over low .. high
        if high <= span:
            seen = (low + high) / 2
        elif low >= span:
            seen = span
        else:
            seen = ((span - low) * (low + span) / 2 + (high - span) * span) / (high - low)
        tokens = c["B"] * seen
        return {"bytes": tokens * token + 4 * tokens / c["page"] + 4 * c["B"] * c["heads"]
                * (c["D"] + 1), "flops": 4 * tokens * c["heads"] * c["D"]}
    if c["kind"] == "append":
        return {"bytes": c["T"] * (4 * c["kv"] * c["D"] + token + 8), "flops": 0}
    # the tables once, and each moved page read and written: the shared last pages of growing
    # sequences, and the live pages behind the number of live pages
    kids = c["parents"] * c["fan"]
    held = c["parents"] * ((c["low"] + c["high"]) / 2 / c["page"] + 0.5)
    live = held + 1.5 * c["parents"] + 0.75 * kids
    moved = kids + live * (1 - live / c["pages"])
    width = c["high"] / c["page"] + 1
    return {"bytes": 2 * moved * c["layers"] * token * c["page"] + 8 * c["pages"]
            + 8 * (c["parents"] + kids) * width, "flops": 0}


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    c = case
    if c["kind"] == "pages":
        return None  # whole numbers and copies
    st = prepare(case, seed)
    if c["kind"] == "w4":
        K, x = c["K"], st["x"].double()
        parts = []
        for n0 in range(0, c["N"], 8192):
            words = st["packed"][n0:n0 + 8192].contiguous().view(torch.int32).long()
            t = torch.zeros(words.shape[0], words.shape[1] * 8, dtype=torch.float64, device=DEV)
            wd = torch.arange(words.shape[1], device=DEV)
            first = wd // 16 * 128 + wd % 4 * 32 + wd % 16 // 4 * 8
            for i in range(8):
                t[:, first + (2 * i if i < 4 else 2 * i - 7)] = \
                    ((words >> (4 * i)) & 15).double() - 8
            s = st["scales"][n0:n0 + 8192].double()
            group = torch.arange(K, device=DEV) // c["group"]
            parts.append(x @ (t[:, :K] * s[:, group]).T)
        return torch.cat(parts, 1)
    meta, layer = st["meta"], st["layers"][0]
    if c["kind"] == "attn":
        G = c["heads"] // c["kv"]
        out = torch.zeros(c["B"], c["heads"], c["D"], dtype=torch.float64, device=DEV)
        lse = torch.full((c["B"], c["heads"]), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(meta["lens"].tolist()):
            j = torch.arange(n, device=DEV)
            if c["window"]:
                j = j[(j < c["sinks"]) | (j >= n - c["window"])]
            if not len(j):
                continue
            p, o = meta["table"][b].long()[j // c["page"]], j % c["page"]
            kv = []
            for w in ("k", "v"):
                x = layer[w][p, :, o].double()
                if layer[w + "_scale"] is not None:
                    x = x / layer[w + "_scale"][p, :, o].double()[..., None]
                kv.append(x)
            for h in range(c["kv"]):
                qs = st["q"][b, h * G:(h + 1) * G].double()
                z = qs @ kv[0][:, h].T / math.sqrt(c["D"])
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
                out[b, h * G:(h + 1) * G] = torch.softmax(z, 1) @ kv[1][:, h]
        return {"out": out, "lse": lse}
    # append: bf16 is a copy; in 8 bits the code is the nearest whole number to x * scale, scale
    # and product being 32-bit numbers by definition (each rounded once here, from 64 bits)
    seqs, pos = st["seqs"].tolist(), st["pos"].tolist()
    if c["dtype"] == "bf16" or c["T"] > 8192:
        return None
    table, got = meta["table"].tolist(), []
    where_p = torch.tensor([table[s][p // c["page"]] for s, p in zip(seqs, pos)], device=DEV)
    where_o = torch.tensor([p % c["page"] for p in pos], device=DEV)
    for w in ("k", "v"):
        held = layer[w].double() / layer[w + "_scale"].double()[..., None]
        x = st[w].double()
        s = (127.0 / x.abs().amax(-1).clamp(min=float(torch.tensor(1e-5)))).float().double()
        q = torch.round((x * s[..., None]).float()).double()
        held[where_p, :, where_o] = q / s[..., None]
        got.append(held)
    return got
