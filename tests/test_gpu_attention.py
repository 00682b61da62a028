"""bitnet_paged_attention against 64-bit attention over the same tokens. The tolerances are those
that decode_ref.attention derives from binary32 arithmetic, plus one rounding to bf16."""
import threading

import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ternary_w2a8_linear_token_b200 as bn
    return bn


def _dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _fill(bn, lens, kv, D, page, dtype, seed=0, layers=1, spare=3):
    """A cache of sequences of these lengths over scattered pages, random tokens everywhere (so a
    token that should not be seen would show)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + spare
    cache = bn.make_cache(P, len(lens), max(max(need), 1) + 1, kv, D, page, layers, dtype)
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    at = 0
    for s, n in enumerate(need):
        cache.table[s, :n] = perm[at:at + n]
        cache.refs[perm[at:at + n].long()] = 1
        at += n
    cache.lens.copy_(_dev(lens))
    for layer in cache.layers:
        for w in range(2):
            x = torch.randn(layer[w].shape, generator=g, device="cuda")
            if dtype == torch.int8:
                layer[w].copy_((x * 40).clamp(-127, 127).round().to(torch.int8))
                layer[2 + w].copy_(torch.rand(layer[2 + w].shape, generator=g, device="cuda") * 60
                                   + 20)
            else:
                layer[w].copy_(x)
    return cache


def _tokens(cache, layer, slot, n):
    """k, v of a slot's n tokens as 64-bit arrays (n, kv_heads, D)."""
    j = torch.arange(n, device="cuda")
    p, o = cache.table[slot].long()[j // cache.page_size], j % cache.page_size
    got = []
    for w in range(2):
        x = cache.layers[layer][w][p, :, o].double()
        if cache.dtype == torch.int8:
            x = x / cache.layers[layer][2 + w][p, :, o].double()[..., None]
        got.append(x.cpu().numpy())
    return got


def _check(cache, q, out, lse, slots=None, scale=None, window=0, sinks=0, layer=0, rows=None):
    qd, got = q.double().cpu().numpy(), out.double().cpu().numpy()
    got_lse = lse.double().cpu().numpy()
    lens = cache.lens.tolist()
    for b in range(q.shape[0]) if rows is None else rows:
        s = b if slots is None else slots[b]
        k, v = _tokens(cache, layer, s, lens[s])
        if window:
            j = np.arange(lens[s])
            seen = (j < sinks) | (j >= lens[s] - window)
            k, v = k[seen], v[seen]
        o, l, to, tl = ref.attention(qd[b], k, v,
                                     cache.head_dim ** -0.5 if scale is None else scale)
        tol = to + ref.BF16_HALF * (np.abs(o) + to)
        err = np.abs(got[b] - o)
        assert np.all(err <= tol), f"query {b} of {lens[s]}: {np.nanmax(err / tol):.2f}"
        if len(k):
            off = np.abs(got_lse[b] - l)
            assert np.all(off <= tl), f"lse {b}: {np.max(off / tl)}"
        else:
            assert np.all(got_lse[b] == -np.inf) and not got[b].any()


def _q(B, heads, D, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(B, heads, D, generator=g, device="cuda").to(torch.bfloat16)


RAGGED = [0, 1, 15, 16, 17, 300, 64, 2, 1025, 0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("D,kv,group", [(128, 5, 4), (64, 2, 1), (128, 1, 8), (64, 1, 16),
                                        (128, 2, 3), (64, 2, 17), (128, 1, 40)])
def test_ragged_batch(bn, D, kv, group, dtype):
    for page in (8, 64):
        cache = _fill(bn, RAGGED, kv, D, page, dtype)
        q = _q(len(RAGGED), kv * group, D)
        out, lse = bn.bitnet_paged_attention(q, cache, return_lse=True)
        _check(cache, q, out, lse)
        again, lse2 = bn.bitnet_paged_attention(q, cache, return_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
        assert cache.errors() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("n", [1, 7, 4096, 33000])
def test_one_sequence(bn, n, dtype):
    """From one token to a length that is split over the whole GPU."""
    cache = _fill(bn, [n], 2, 128, 16, dtype)
    q = _q(1, 8, 128)
    _check(cache, q, *bn.bitnet_paged_attention(q, cache, return_lse=True))


def test_one_long_among_many_short(bn):
    lens = [5] * 100 + [20001] + [40] * 60
    cache = _fill(bn, lens, 2, 64, 32, torch.bfloat16)
    q = _q(len(lens), 8, 64)
    _check(cache, q, *bn.bitnet_paged_attention(q, cache, return_lse=True))


@pytest.mark.parametrize("many", [300, 2500])
def test_many_sequences(bn, many):
    """More sequences than CTAs, and than one round of the search over lengths."""
    lens = [(i * 37) % 50 for i in range(many)]
    cache = _fill(bn, lens, 1, 64, 16, torch.bfloat16)
    q = _q(many, 2, 64)
    _check(cache, q, *bn.bitnet_paged_attention(q, cache, return_lse=True))


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (100, 0), (64, 70), (5000, 3),
                                          (2 ** 40, 2 ** 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_window_and_sinks(bn, window, sinks, dtype):
    lens = RAGGED + [2000, 135, 134, 133]
    cache = _fill(bn, lens, 2, 128, 16, dtype)
    q = _q(len(lens), 8, 128)
    out, lse = bn.bitnet_paged_attention(q, cache, window=window, sinks=sinks, return_lse=True)
    _check(cache, q, out, lse, window=window, sinks=sinks)


def test_hidden_tokens_may_hold_anything(bn):
    """Inf and NaN behind the end of a sequence, in pages of nobody and outside the window, and
    page numbers that no visible token needs."""
    for dtype in (torch.bfloat16, torch.int8):
        lens = [21, 100, 300]
        cache = _fill(bn, lens, 2, 64, 16, dtype)
        q = _q(3, 8, 64)
        want, want_lse = bn.bitnet_paged_attention(q, cache, window=40, sinks=2, return_lse=True)
        k, v = cache.layers[0][:2]
        seen = torch.zeros(k.shape[0], 16, dtype=torch.bool)
        table = cache.table.cpu()
        for s, n in enumerate(lens):
            for j in range(n):
                if j < 2 or j >= n - 40:
                    seen[table[s, j // 16], j % 16] = True
        hide = ~seen.cuda()
        bad = [k, v] if dtype == torch.bfloat16 else list(cache.layers[0][2:])
        for i, t in enumerate(bad):
            t.transpose(1, 2)[hide] = (float("nan"), float("inf"))[i]
        cache.table[2, 3:10] = 10 ** 9  # hidden pages of a long sequence
        cache.table[0, 2:] = -5  # entries behind the end
        out, lse = bn.bitnet_paged_attention(q, cache, window=40, sinks=2, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert cache.errors() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_nan_in_sight_shows(bn, dtype):
    """A NaN in q, or in a visible token, comes out where the formula has one and nowhere else: in
    items of one CTA and in ones that several CTAs share."""
    cache = _fill(bn, [21, 4000], 2, 64, 16, dtype)
    q = _q(2, 8, 64)
    for b in range(2):  # one dimension of one query head
        bad = q.clone()
        bad[b, 3, 5] = float("nan")
        out, lse = bn.bitnet_paged_attention(bad, cache, return_lse=True)
        assert out[b, 3].isnan().all() and lse[b, 3].isnan()
        clean, clean_lse = bn.bitnet_paged_attention(q, cache, return_lse=True)
        out[b, 3], lse[b, 3] = clean[b, 3], clean_lse[b, 3]
        _check(cache, q, out, lse)
    for w in range(2):  # a token of key/value head 1 (query heads 4 to 7), of K or of V
        for s, j in ((0, 20), (1, 2345)):
            at = (int(cache.table[s, j // 16]), 1, j % 16)
            pool, i = (cache.layers[0][w], at + (7,)) if dtype == torch.bfloat16 else \
                (cache.layers[0][2 + w], at)
            keep = pool[i].item()
            pool[i] = float("nan")
            out, lse = bn.bitnet_paged_attention(q, cache, return_lse=True)
            pool[i] = keep
            want = torch.zeros_like(out, dtype=torch.bool)
            want[s, 4:, slice(7, 8) if w and dtype == torch.bfloat16 else slice(None)] = True
            assert torch.equal(out.isnan(), want)
            want = torch.zeros_like(lse, dtype=torch.bool)
            want[s, 4:] = w == 0
            assert torch.equal(lse.isnan(), want)


def test_bad_pages_and_slots_are_skipped_and_reported(bn):
    lens = [40, 70, 0]
    cache = _fill(bn, lens, 2, 64, 16, torch.bfloat16)
    q = _q(5, 8, 64)
    keep = cache.table.clone()
    cache.table[1, 1] = cache.num_pages
    cache.table[1, 3] = -1
    slots = [1, -1, 0, 3, 2]
    out = torch.full_like(q, 9.0)
    lse = torch.full((5, 8), 9.0, device="cuda")
    bn.bitnet_paged_attention(q, cache, seqs=_dev(slots), out=out, lse=lse)
    assert cache.errors() == bn.CACHE_ERR_PAGE | bn.CACHE_ERR_SEQ
    for b in (1, 3):  # skipped queries leave their rows
        assert torch.all(out[b] == 9.0) and torch.all(lse[b] == 9.0)
    cache.table.copy_(keep)
    _check(cache, q, out, lse, slots, rows=[2, 4])
    k, v = _tokens(cache, 0, 1, 70)
    there = np.array([j // 16 not in (1, 3) for j in range(70)])
    o, l, to, tl = ref.attention(q[0].double().cpu().numpy(), k[there], v[there], 64 ** -0.5)
    assert np.all(np.abs(out[0].double().cpu().numpy() - o)
                  <= to + ref.BF16_HALF * (np.abs(o) + to))
    # a length outside the table is cut at the table's end
    full = cache.max_pages * 16
    cache2 = _fill(bn, [full], 2, 64, 16, torch.bfloat16)
    cache2.table[0, -1] = cache2.table[0, 0]
    q2 = _q(1, 8, 64)
    cap = cache2.max_pages * 16
    cache2.lens.fill_(cap)
    want = bn.bitnet_paged_attention(q2, cache2)
    cache2.lens.fill_(cap + 1)
    got = bn.bitnet_paged_attention(q2, cache2)
    assert cache2.errors() == bn.CACHE_ERR_LEN and torch.equal(got, want)
    cache2.lens.fill_(-1)
    got, lse = bn.bitnet_paged_attention(q2, cache2, return_lse=True)
    assert cache2.errors() == bn.CACHE_ERR_LEN and not got.any() and torch.all(lse == -np.inf)


@pytest.mark.parametrize("scale", [1.0, 5.0, -0.3, 0.0])
def test_scales_and_peaked_scores(bn, scale):
    cache = _fill(bn, [500, 33, 1], 2, 128, 16, torch.bfloat16)
    q = _q(3, 8, 128)
    _check(cache, q, *bn.bitnet_paged_attention(q, cache, scale=scale, return_lse=True),
           scale=scale)


def test_scores_far_from_zero(bn):
    """Scores of several thousand, rising along the sequence (every step changes the maximum)."""
    cache = _fill(bn, [257], 1, 64, 16, torch.bfloat16)
    q = torch.ones(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    for j in range(257):
        cache.layers[0][0][cache.table[0, j // 16], 0, j % 16] = float(j - 128)
    _check(cache, q, *bn.bitnet_paged_attention(q, cache, scale=0.5, return_lse=True), scale=0.5)


def test_shapes_slots_and_layers(bn):
    """Flat queries, the same slot twice, several layers, no lse."""
    cache = _fill(bn, [90, 5, 31], 2, 64, 8, torch.bfloat16, layers=2)
    q = _q(4, 6, 64)
    slots = [2, 0, 2, 1]
    out, lse = bn.bitnet_paged_attention(q.view(4, -1), cache, 1, seqs=_dev(slots), return_lse=True)
    assert out.shape == (4, 6 * 64)
    _check(cache, q, out.view(4, 6, 64), lse, slots, layer=1)
    alone = bn.bitnet_paged_attention(q, cache, 1, seqs=_dev(slots))
    assert torch.equal(alone.view(4, -1), out)


def test_offsets_past_32_bits(bn):
    """A pool of more than 2^31 values: its last pages are read and written at the right place."""
    page, kv, D = 256, 8, 128
    P = (1 << 31) // (page * kv * D) + 3
    cache = bn.make_cache(P, 2, 3, kv, D, page)
    cache.table[0, :3] = _dev([P - 1, 0, P - 2])
    cache.refs[torch.tensor([P - 1, 0, P - 2], device="cuda")] = 1
    cache.lens[0] = 700
    g = torch.Generator(device="cuda").manual_seed(3)
    kv_new = [torch.randn(700, kv, D, generator=g, device="cuda").to(torch.bfloat16)
              for _ in range(2)]
    bn.bitnet_cache_append(cache, 0, *kv_new, _dev([0] * 700), _dev(list(range(700))))
    assert torch.equal(cache.layers[0][0][P - 1].transpose(0, 1), kv_new[0][:256])
    q = _q(1, 16, D)
    _check(cache, q, *bn.bitnet_paged_attention(q, cache, seqs=_dev([0]), return_lse=True))
    bn.bitnet_cache_copy(cache, _dev([1, 0, P - 1, P - 3]))
    assert torch.equal(cache.layers[0][1][P - 3], cache.layers[0][1][P - 1])


def test_two_captured_graphs_with_their_own_workspaces(bn):
    """Captured once, replayed after the sequences have grown, two graphs in turn."""
    lens = [60, 1, 200]
    cache = _fill(bn, lens, 2, 128, 16, torch.bfloat16, spare=40)
    cache.table.copy_(torch.arange(cache.table.numel(), device="cuda").view_as(cache.table)
                      % cache.num_pages)
    qs = [_q(3, 8, 128, s) for s in (1, 2)]
    graphs = []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = bn.bitnet_paged_attention(q, cache, return_lse=True)
        graphs.append((g, r))
    for step in range(3):
        cache.lens.copy_(_dev([60 + 5 * step, 1 + step, 200 + 8 * step]))
        for (g, _) in graphs:
            g.replay()
        torch.cuda.synchronize()
        for q, (_, r) in zip(qs, graphs):
            _check(cache, q, *r)


def test_side_stream(bn):
    cache = _fill(bn, [900, 30], 2, 128, 16, torch.int8)
    q = _q(2, 8, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = bn.bitnet_paged_attention(q, cache, return_lse=True, stream=side)
    side.synchronize()
    _check(cache, q, out, lse)


def test_workspace_contents_do_not_matter(bn):
    """A workspace of exactly the size asked for, full of ones and of an earlier call's leavings."""
    g = torch.Generator(device="cuda").manual_seed(9)
    results = []
    size = 0
    for kind in range(3):
        cache = _fill(bn, [700, 0, 33, 5000], 2, 128, 16, torch.bfloat16)
        q = _q(4, 8, 128)
        size = cache.attention_workspace_size(4, 8)
        buf = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
        ws = buf[:size]
        if kind == 1:
            other = _fill(bn, [9000] * 4, 2, 128, 16, torch.bfloat16, seed=4)
            bn.bitnet_paged_attention(q, other, workspace=ws)
        elif kind == 2:
            ws.copy_(torch.randint(0, 256, (size,), generator=g, device="cuda").to(torch.uint8))
        out, lse = bn.bitnet_paged_attention(q, cache, workspace=ws, return_lse=True)
        _check(cache, q, out, lse)
        results.append((out, lse))
        assert torch.all(buf[size:] == 255)
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(r, results[0]))
    with pytest.raises(bn.BitnetError) as e:
        bn.bitnet_paged_attention(q, cache, workspace=ws[:-1].clone())
    assert e.value.status == bn.ERR_WORKSPACE


def test_calls_at_once_on_two_streams(bn):
    caches = [_fill(bn, [3000, 17, 800], 2, 128, 16, torch.bfloat16, seed=s) for s in (1, 2)]
    qs = [_q(3, 8, 128, s) for s in (3, 4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(bn.bitnet_paged_attention(qs[i], caches[i], return_lse=True,
                                                    stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        _check(caches[i], qs[i], *got[i][0])
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, got[i][0]))


def test_more_queries_than_one_look_with_gaps(bn):
    """Padded entries between and behind the queries of a batch of several hundred."""
    lens = [(i * 53) % 300 for i in range(90)]
    cache = _fill(bn, lens, 2, 64, 32, torch.int8)
    slots = [(i * 7) % 90 if i % 5 else -1 for i in range(400)] + [-1] * 150
    q = _q(len(slots), 4, 64)
    out = torch.full_like(q, 3.0)
    lse = torch.full((len(slots), 4), 3.0, device="cuda")
    bn.bitnet_paged_attention(q, cache, seqs=_dev(slots), out=out, lse=lse)
    rows = [b for b, s in enumerate(slots) if s >= 0]
    _check(cache, q, out, lse, slots, rows=rows)
    rest = [b for b, s in enumerate(slots) if s < 0]
    assert torch.all(out[rest] == 3.0) and torch.all(lse[rest] == 3.0)
    out.fill_(3.0)
    bn.bitnet_paged_attention(q, cache, seqs=_dev([-1] * len(slots)), out=out)
    assert torch.all(out == 3.0) and cache.errors() == 0


def test_misaligned_and_foreign_tensors_are_refused(bn):
    cache = _fill(bn, [20], 2, 64, 16, torch.bfloat16)
    q = _q(1, 4, 64)
    with pytest.raises(bn.BitnetError) as e:
        buf = torch.zeros(257, dtype=torch.bfloat16, device="cuda")
        bn.bitnet_paged_attention(buf[1:].view(1, 4, 64), cache)
    assert e.value.status == bn.ERR_ALIGN
    for bad in (q.float(), q.cpu(), q[:, :, :32], q.transpose(1, 2), _q(2, 4, 64)):
        with pytest.raises((ValueError, bn.BitnetError)):
            bn.bitnet_paged_attention(bad, cache)
    with pytest.raises(bn.BitnetError):
        bn.bitnet_paged_attention(_q(1, 3, 64), cache)  # 3 heads over 2
    with pytest.raises(IndexError):
        bn.bitnet_paged_attention(q, cache, 1)


def test_default_stream_shares_scratch_and_others_do_not(bn):
    """Calls on the default stream, on a side stream and in a captured graph, interleaved: the
    default stream's kept workspace is nobody else's."""
    cache = _fill(bn, [6000, 40], 2, 128, 16, torch.bfloat16)
    qs = [_q(2, 8, 128, s) for s in (1, 2, 3)]
    want = [bn.bitnet_paged_attention(q, cache) for q in qs]
    small = bn.bitnet_paged_attention(qs[0][:1], cache, seqs=_dev([1]))
    kept = cache._kept.ws
    assert kept is not None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = bn.bitnet_paged_attention(qs[1], cache)
    assert cache._kept.ws is kept
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            graph.replay()
        a = bn.bitnet_paged_attention(qs[0], cache)
        b = bn.bitnet_paged_attention(qs[2], cache, stream=side)
        c = bn.bitnet_paged_attention(qs[0][:1], cache, seqs=_dev([1]))
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[2]) and torch.equal(c, small)
        assert torch.equal(captured, want[1])
    assert cache._kept.ws is kept


def test_two_threads_on_the_default_stream(bn):
    """Their calls may mix on the stream; each thread has a workspace of its own."""
    cache = _fill(bn, [9000, 700], 2, 128, 16, torch.bfloat16)
    qs = [_q(2, 8, 128, s) for s in (1, 2)]
    want = [bn.bitnet_paged_attention(q, cache, return_lse=True) for q in qs]
    wrong = []

    def work(i):
        for _ in range(200):
            got = bn.bitnet_paged_attention(qs[i], cache, return_lse=True)
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_tensors_of_a_call_on_another_stream_live_long_enough(bn):
    """With stream given: what the caller drops after the call, and what the call allocates while
    the current stream still works on memory that it has given back."""
    cache = _fill(bn, [300, 77], 2, 64, 16, torch.int8)
    q = _q(2, 8, 64)
    want = bn.bitnet_paged_attention(q, cache)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        early = q.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        out = bn.bitnet_paged_attention(early, cache, stream=side)
        del early
        junk = [torch.full_like(q, 9.0) for _ in range(8)]  # the dropped query's memory, if free
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del junk, out
        late = torch.empty_like(q)
        torch.cuda._sleep(20_000_000)
        late.fill_(9.0)
        del late  # free for the current stream, which has yet to write it
        out = bn.bitnet_paged_attention(q, cache, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del out


def test_captured_with_a_stream_given(bn):
    """A captured step whose calls name their stream: the capture's own, and one forked off it."""
    cache = _fill(bn, [40, 700], 2, 64, 16, torch.bfloat16, spare=20)
    seqs, one = _dev([0, 1]), _dev([1, 1])
    q, k, v = _q(2, 8, 64), _q(2, 2, 64, 2), _q(2, 2, 64, 3)
    packed, scales = bn.bitnet_pack_w4(torch.randn(96, 512, device="cuda"))
    flat = q.view(2, 512)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    lens = cache.lens.tolist()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        copies = bn.bitnet_cache_extend(cache, seqs, one, stream=here)
        bn.bitnet_cache_copy(cache, copies, stream=here)
        bn.bitnet_cache_append(cache, 0, k, v, seqs, stream=here)
        side.wait_stream(here)
        y = bn.bitnet_linear_w4(flat, packed, scales, 128, stream=side)
        out, lse = bn.bitnet_paged_attention(q, cache, seqs=seqs, return_lse=True, stream=side)
        here.wait_stream(side)
    assert cache.lens.tolist() == lens
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert cache.errors() == 0 and cache.lens.tolist() == [n + 5 for n in lens]
    _check(cache, q, out, lse)
    assert torch.equal(y, bn.bitnet_linear_w4(flat, packed, scales, 128))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_weights_keep_all_their_bits(bn, dtype):
    """Weights 1, 1 and w of three tokens whose values cancel all but w's last bits: v = -p1, -p2 and
    1, where p1 + p2 are the first 14 bits of w (8-bit codes times powers of two, exact in either
    type), so out = (w - p1 - p2) / (2 + w), about 2^-16. Against the formula in 64 bits: the score
    and its exponential are off by (4 |z| + 6) binary32 steps of w, as decode_ref derives them, the
    six terms and two joins of the sum by eight steps of its largest part; then one rounding."""
    B, kv, D = 64, 8, 64
    cache = _fill(bn, [3] * B, kv, D, 16, dtype)
    layer = cache.layers[0]
    g = np.random.default_rng(12)
    z = -ref.bf16(g.uniform(0.02, 0.68, (B, kv))).double().numpy()
    w = np.exp(z)
    p1 = np.floor(w * 128) / 128
    p2 = np.floor((w - p1) * 2.0 ** 14) / 2.0 ** 14
    k, v = np.zeros((B, kv, 3, D)), np.zeros((B, kv, 3, D))
    k[:, :, 2, 0] = 1.0
    v[:, :, 0], v[:, :, 1], v[:, :, 2] = -p1[..., None], -p2[..., None], 1.0
    for pool, x in zip(range(2), (k, v)):
        page = cache.table[:, 0].long()
        x = torch.from_numpy(x).cuda()
        if dtype == torch.int8:
            scale = torch.tensor([2.0 ** 7, 2.0 ** 14, 1.0] if pool else [1.0] * 3, device="cuda",
                                 dtype=torch.float64)
            layer[pool][page, :, :3] = (x * scale[:, None]).to(torch.int8)
            layer[2 + pool][page, :, :3] = scale.float().expand(B, kv, 3)
        else:
            layer[pool][page, :, :3] = x.to(torch.bfloat16)
            assert torch.equal(layer[pool][page, :, :3].double(), x)
    q = torch.zeros(B, kv, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = torch.from_numpy(z).cuda()
    out = bn.bitnet_paged_attention(q, cache, scale=1.0).double().cpu().numpy()
    want = ((w - p1 - p2) / (2 + w))[..., None]
    tol = (((4 * np.abs(z) + 6) * w + 8) * ref.F32_STEP / (2 + w))[..., None]
    tol = tol + ref.BF16_HALF * (np.abs(want) + tol)
    err = np.abs(out - want)
    assert np.all(err <= tol), f"{np.max(err / tol):.2f} of the tolerance"
    assert np.median(np.abs(want) / tol) > 4  # (what cancels is large beside it)


@pytest.mark.parametrize("far", [8, 20, 60, 100])
@pytest.mark.parametrize("kv,group", [(2, 4), (1, 12)])
def test_queries_of_a_wide_range_over_8_bits(bn, kv, group, far):
    """Small values of q count in full beside one 2^far times as large that meets codes of zero, and
    beside one that meets others."""
    cache = _fill(bn, [40, 700], kv, 64, 16, torch.int8)
    q = (_q(2, kv * group, 64).float() * 2.0 ** -far).to(torch.bfloat16)
    q[:, :, 5] = 1.0
    q[1, 0, 9] = 0.0
    for layer in cache.layers:
        layer[0][..., 5] = 0
    scale = 0.125 * 2.0 ** far
    _check(cache, q, *bn.bitnet_paged_attention(q, cache, scale=scale, return_lse=True),
           scale=scale)
    q[:, :, 5] *= 2.0 ** (3 - far)
    cache.layers[0][0][..., 5] = -3
    _check(cache, q, *bn.bitnet_paged_attention(q, cache, scale=scale, return_lse=True),
           scale=scale)


@pytest.mark.parametrize("D,kv,group", [(64, 2, 4), (128, 1, 12)])
def test_scores_of_minus_infinity(bn, D, kv, group):
    """Inf in K against a q of the other sign. All visible scores -inf: out is the formula's 0 / 0 and
    lse its log 0, in an item of one CTA, one that several share, and a window of one token; with a
    q of the same sign NaN in both. Where some scores are finite, attention over their tokens alone.
    Without a visible token (no tokens, or only pages outside the pool) out stays 0."""
    lens = [1, 40, 5000, 5000, 17, 0, 33]
    cache = _fill(bn, lens, kv, D, 16, torch.bfloat16)
    k = cache.layers[0][0]
    q = _q(len(lens), kv * group, D)
    q[..., 3] = torch.where(torch.arange(kv * group, device="cuda") % 2 == 1, 0.5, -0.5)

    def pages(s, n):
        return cache.table[s, :n].long()

    for s in (0, 1, 2):
        k[pages(s, -(-lens[s] // 16)), :, :, 3] = float("inf")
    k[pages(3, 200), :, :, 3] = float("inf")  # 3200 of 5000 tokens
    k[pages(4, 1), :, :, 3] = float("-inf")  # 16 of 17
    cache.table[6, :3] = -1
    down = torch.arange(kv * group, device="cuda") % 2 == 0
    out, lse = bn.bitnet_paged_attention(q, cache, return_lse=True)
    assert cache.errors() == bn.CACHE_ERR_PAGE
    assert out[:3].isnan().all()
    assert torch.all(lse[:3, down] == -np.inf) and lse[:3, ~down].isnan().all()
    assert not out[5:].any() and torch.all(lse[5:] == -np.inf)
    for s, first, heads in ((3, 3200, down), (4, 16, ~down)):
        assert out[s, ~heads].isnan().all() and lse[s, ~heads].isnan().all()
        kk, vv = _tokens(cache, 0, s, lens[s])
        o, l, to, tl = ref.attention(q[s].double().cpu().numpy(), kk[first:], vv[first:], D ** -0.5)
        h = heads.cpu().numpy()
        tol = to + ref.BF16_HALF * (np.abs(o) + to)
        assert np.all(np.abs(out[s].double().cpu().numpy() - o)[h] <= tol[h])
        assert np.all(np.abs(lse[s].double().cpu().numpy() - l)[h] <= tl[h])
    one, lse1 = bn.bitnet_paged_attention(q[1:3], cache, seqs=_dev([1, 2]), window=1,
                                          return_lse=True)
    assert one.isnan().all() and torch.all(lse1[:, down] == -np.inf)


def test_scores_that_overflow(bn):
    """Finite values whose scores pass binary32's range downwards are not taken for no token at all."""
    cache = _fill(bn, [3, 900], 1, 64, 16, torch.bfloat16)
    cache.layers[0][0].fill_(1e30)
    q = torch.full((2, 2, 64), -1e30, dtype=torch.bfloat16, device="cuda")
    out, lse = bn.bitnet_paged_attention(q, cache, return_lse=True)
    assert out.isnan().all() and torch.all(lse == -np.inf)
