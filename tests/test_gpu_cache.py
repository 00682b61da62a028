"""The paged cache's calls against a model of plain Python lists: all results are whole numbers
or copies and have to be equal."""
import random

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


def _make(bn, P, S, W, page, layers=1, dtype=torch.bfloat16, kv=2, D=64):
    cache = bn.make_cache(P, S, W, kv, D, page, layers, dtype)
    return cache, ref.Model(P, S, W, page)


@pytest.mark.parametrize("page", [8, 16, 256])
def test_a_long_life(bn, page):
    """Random forks, extensions, frees and compactions of a small pool, step by step."""
    rng = random.Random(page)
    cache, m = _make(bn, 97, 12, 6, page)
    full = 0
    for step in range(120):
        slots = list(range(12))
        rng.shuffle(slots)
        what = rng.choice(["fork", "extend", "extend", "free", "compact"])
        if what == "fork":
            dst = [s for s in slots if m.lens[s] == 0][:rng.randint(1, 3)]
            src = [rng.choice([s for s in slots if s not in dst] or [0]) for _ in dst]
            if not dst:
                continue
            if rng.random() < 0.3:
                src, dst = src + [-1, 0], dst + [5, -3]  # padding on either side
                dst[-2] = 5 if 5 not in dst[:-2] else -1
            bn.bitnet_cache_fork(cache, _dev(src), _dev(dst))
            m.fork(src, dst)
        elif what == "extend":
            seqs = slots[:rng.randint(1, 12)]
            add = [rng.choice([0, 1, 1, page, rng.randint(0, 2 * page)]) for _ in seqs]
            add = [min(a, 6 * page - m.lens[s]) for s, a in zip(seqs, add)]
            if rng.random() < 0.3:
                seqs, add = seqs + [-1], add + [3]
            copies = bn.bitnet_cache_extend(cache, _dev(seqs), _dev(add))
            want = m.extend(seqs, add)
            if want is None:
                full += 1
                assert cache.errors() == bn.CACHE_ERR_FULL and ref.pairs(copies) == []
            else:
                assert ref.pairs(copies) == want
        elif what == "free":
            seqs = slots[:rng.randint(1, 4)] + [-7]
            bn.bitnet_cache_free(cache, _dev(seqs))
            m.free(seqs)
        else:
            assert ref.pairs(bn.bitnet_cache_compact(cache)) == m.compact()
        m.check(cache)
        assert cache.errors() == 0
    assert all(r >= 0 for r in m.refs)


def test_full_changes_nothing(bn):
    cache, m = _make(bn, 10, 4, 8, 16)
    copies = bn.bitnet_cache_extend(cache, _dev([0, 1]), _dev([100, 30]))
    assert m.extend([0, 1], [100, 30]) == ref.pairs(copies) == []
    bn.bitnet_cache_fork(cache, _dev([1]), _dev([2]))
    m.fork([1], [2])
    m.check(cache)
    copies = bn.bitnet_cache_extend(cache, _dev([2, 3]), _dev([1, 16]))  # one page left, two needed
    assert cache.errors() == bn.CACHE_ERR_FULL and ref.pairs(copies) == []
    m.check(cache)
    copies = bn.bitnet_cache_extend(cache, _dev([2]), _dev([1]))
    assert ref.pairs(copies) == m.extend([2], [1]) == [(8, 9)]
    m.check(cache)
    assert cache.errors() == 0


def test_all_holders_grow_and_the_last_keeps_the_page(bn):
    cache, m = _make(bn, 64, 8, 4, 16)
    bn.bitnet_cache_extend(cache, _dev([3]), _dev([20]))
    m.extend([3], [20])
    src, dst = [3, 3, 3], [0, 1, 2]
    bn.bitnet_cache_fork(cache, _dev(src), _dev(dst))
    m.fork(src, dst)
    copies = bn.bitnet_cache_extend(cache, _dev([1, 3, 0, 2]), _dev([1, 1, 0, 1]))
    want = m.extend([1, 3, 0, 2], [1, 1, 0, 1])  # slot 0 stays, so everybody copies
    assert ref.pairs(copies) == want and len(want) == 3
    m.check(cache)
    src, dst = [3, 3], [5, 6]
    bn.bitnet_cache_fork(cache, _dev(src), _dev(dst))
    m.fork(src, dst)
    copies = bn.bitnet_cache_extend(cache, _dev([5, 6, 3]), _dev([2, 2, 2]))
    want = m.extend([5, 6, 3], [2, 2, 2])
    assert ref.pairs(copies) == want and len(want) == 2  # slot 3, the last, keeps it
    m.check(cache)


@pytest.mark.parametrize("P,n", [(40000, 1500), (70001, 2100)])
def test_many_pages_and_sequences(bn, P, n):
    """More pages than one round of the scan, more entries than threads, long prompts."""
    rng = random.Random(P)
    cache, m = _make(bn, P, 2 * n, 64, 8, kv=1)
    seqs = rng.sample(range(n), n)
    add = [rng.randint(0, 200) for _ in seqs]
    assert ref.pairs(bn.bitnet_cache_extend(cache, _dev(seqs), _dev(add))) == m.extend(seqs, add)
    m.check(cache)
    src, dst = [rng.randrange(n) for _ in range(n)], list(range(n, 2 * n))
    bn.bitnet_cache_fork(cache, _dev(src), _dev(dst))
    m.fork(src, dst)
    m.check(cache)
    seqs = rng.sample(range(2 * n), 2 * n)
    add = [rng.randint(0, 9) for _ in seqs]
    assert ref.pairs(bn.bitnet_cache_extend(cache, _dev(seqs), _dev(add))) == m.extend(seqs, add)
    m.check(cache)
    gone = rng.sample(range(2 * n), n)
    bn.bitnet_cache_free(cache, _dev(gone))
    m.free(gone)
    m.check(cache)
    assert ref.pairs(bn.bitnet_cache_compact(cache)) == m.compact()
    m.check(cache)
    assert cache.errors() == 0


def test_device_checks_change_nothing(bn):
    cache, m = _make(bn, 32, 4, 4, 16)
    bn.bitnet_cache_extend(cache, _dev([0, 1]), _dev([20, 5]))
    m.extend([0, 1], [20, 5])
    SEQ, LEN, PAGE = bn.CACHE_ERR_SEQ, bn.CACHE_ERR_LEN, bn.CACHE_ERR_PAGE
    for bits, call in [
            (SEQ, lambda: bn.bitnet_cache_fork(cache, _dev([0]), _dev([4]))),
            (SEQ, lambda: bn.bitnet_cache_fork(cache, _dev([4]), _dev([2]))),
            (SEQ, lambda: bn.bitnet_cache_fork(cache, _dev([0]), _dev([1]))),  # not empty
            (SEQ, lambda: bn.bitnet_cache_fork(cache, _dev([0, 1]), _dev([2, 2]))),
            (SEQ, lambda: bn.bitnet_cache_free(cache, _dev([1, 1]))),
            (SEQ, lambda: bn.bitnet_cache_free(cache, _dev([1, 99]))),
            (SEQ, lambda: bn.bitnet_cache_extend(cache, _dev([2, 0, 2]), _dev([1, 1, 1]))),
            (SEQ, lambda: bn.bitnet_cache_extend(cache, _dev([1, 1 << 30]), _dev([1, 1]))),
            (LEN, lambda: bn.bitnet_cache_extend(cache, _dev([0, 1]), _dev([1, -1]))),
            (LEN, lambda: bn.bitnet_cache_extend(cache, _dev([1, 0]), _dev([1, 45]))),
            (LEN, lambda: bn.bitnet_cache_extend(cache, _dev([1]), _dev([2 ** 31 - 1]))),
    ]:
        got = call()
        assert cache.errors() == bits
        if got is not None:
            assert ref.pairs(got) == []
        m.check(cache)
    # a bad page of a shared row is reported, and the pool's other counts stay right
    cache.table[0, 1] = 32
    bn.bitnet_cache_fork(cache, _dev([0]), _dev([2]))
    assert cache.errors() == PAGE
    assert cache.refs.tolist() == [2, 1, 1] + [0] * 29
    bn.bitnet_cache_free(cache, _dev([2, 0]))
    assert cache.errors() == PAGE
    assert cache.refs.tolist() == [0, 1, 1] + [0] * 29


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("D,kv,page", [(64, 1, 8), (128, 5, 16), (64, 3, 256)])
def test_append_and_copy(bn, D, kv, page, dtype):
    """Tokens go where the table says, in the quantiser's codes; copied pages are equal in every
    layer, and all other pages stay."""
    g = np.random.default_rng([D, kv, page])
    cache, m = _make(bn, 40, 6, 5, page, 2, dtype, kv, D)
    lens = [0, 1, page, page + 3, 2 * page - 1, 4 * page]
    bn.bitnet_cache_extend(cache, _dev(list(range(6))), _dev(lens))
    m.extend(list(range(6)), lens)
    tokens = [(s, p) for s in range(6) for p in range(lens[s])]
    random.Random(1).shuffle(tokens)
    skip = len(tokens) // 3
    tokens[skip] = (-1, 0)  # a padded entry
    x = [ref.bf16(g.standard_normal((len(tokens), kv, D))) for _ in range(2)]
    x[0][0] = 0.0  # a token of zeros
    pools = [[t.clone() for t in layer] for layer in cache.layers]
    bn.bitnet_cache_append(cache, 1, x[0].cuda(), x[1].view(len(tokens), -1).cuda(),
                           _dev([s for s, _ in tokens]), _dev([p for _, p in tokens]))
    for t, (s, p) in enumerate(tokens):
        if s < 0:
            continue
        page_no, off = m.table[s][p // page], p % page
        for w in range(2):
            if dtype == torch.int8:
                q, sc = ref.quantise(x[w][t])
                pools[1][w][page_no, :, off] = torch.from_numpy(q).cuda()
                pools[1][2 + w][page_no, :, off] = torch.from_numpy(sc).cuda()
            else:
                pools[1][w][page_no, :, off] = x[w][t].cuda()
    for got, want in zip(cache.layers, pools):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    # one new token each, by default in the last place of slots 0 .. T - 1
    extra = [ref.bf16(g.standard_normal((6, kv, D))).cuda() for _ in range(2)]
    bn.bitnet_cache_extend(cache, _dev([0]), _dev([1]))
    bn.bitnet_cache_append(cache, 0, *extra)
    table, last = cache.table.tolist(), cache.lens.tolist()
    for s in range(6):
        got = cache.layers[0][0][table[s][(last[s] - 1) // page], :, (last[s] - 1) % page]
        if dtype == torch.int8:
            q, _ = ref.quantise(extra[0][s].cpu())
            assert np.array_equal(got.cpu().numpy(), q)
        else:
            assert torch.equal(got, extra[0][s])
    pools = [[t.clone() for t in layer] for layer in cache.layers]
    moves = [(3, 30), (0, 39), (5, 25)]
    copies = _dev([3, 0] + [v for pr in moves for v in pr] + [9, 9, 9, 9])
    bn.bitnet_cache_copy(cache, copies)
    for got, want in zip(cache.layers, pools):
        for a, b in zip(got, want):
            for f, t in moves:
                b[t] = b[f]
            assert torch.equal(a, b)
    assert cache.errors() == 0


def test_append_and_copy_report_what_they_skip(bn):
    cache, _ = _make(bn, 8, 3, 2, 16)
    bn.bitnet_cache_extend(cache, _dev([0, 1]), _dev([16, 3]))
    before = cache.layers[0][0].clone()
    x = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    for seq, pos, bits in [(0, 16, bn.CACHE_ERR_LEN), (1, 3, bn.CACHE_ERR_LEN),
                           (1, -1, bn.CACHE_ERR_LEN), (2, 0, bn.CACHE_ERR_LEN),
                           (3, 0, bn.CACHE_ERR_SEQ)]:
        bn.bitnet_cache_append(cache, 0, x, x, _dev([seq]), _dev([pos]))
        assert cache.errors() == bits
    cache.table[1, 0] = 8
    bn.bitnet_cache_append(cache, 0, x, x, _dev([1]), _dev([0]))
    assert cache.errors() == bn.CACHE_ERR_PAGE
    cache.table[1, 0] = -1
    bn.bitnet_cache_append(cache, 0, x, x, _dev([1]), _dev([0]))
    assert cache.errors() == bn.CACHE_ERR_PAGE
    assert torch.equal(before, cache.layers[0][0])
    cache.layers[0][0][2] = 1.0
    bn.bitnet_cache_copy(cache, _dev([3, 0, 2, 8, -1, 3, 2, 5]))
    assert cache.errors() == bn.CACHE_ERR_PAGE
    assert [bool(cache.layers[0][0][p].any()) for p in range(8)] == [False] * 2 + [True] + \
        [False] * 2 + [True] + [False] * 2
    bn.bitnet_cache_copy(cache, _dev([100, 0, 2, 6]))  # a count past the list is cut
    assert cache.errors() == 0 and bool(cache.layers[0][0][6].all())


def test_quantised_ties(bn):
    """Values at half steps round to even, as bitnet_quant_act rounds them."""
    cache, _ = _make(bn, 2, 1, 1, 16, dtype=torch.int8, kv=1)
    bn.bitnet_cache_extend(cache, _dev([0]), _dev([1]))
    x = torch.zeros(1, 1, 64)
    x[0, 0, :7] = torch.tensor([127.0, 0.5, 1.5, -2.5, -127.0, 63.5, 126.5])
    x = x.to(torch.bfloat16)
    bn.bitnet_cache_append(cache, 0, x.cuda(), (x * 2).cuda())
    for w, s in ((0, 1.0), (1, 0.5)):
        q, sc = ref.quantise((x * (w + 1))[0])
        assert np.array_equal(cache.layers[0][w][0, :, 0].cpu().numpy(), q)
        assert cache.layers[0][2 + w][0, 0, 0].item() == s == sc[0]


def test_more_slots_than_the_bitmap(bn):
    """Duplicates are found in caches of more slots than one CTA keeps marks for."""
    cache, m = _make(bn, 50, 200000, 2, 16, kv=1)
    seqs, add = [199999, 5, 131072, 131071], [3, 20, 1, 32]
    assert ref.pairs(bn.bitnet_cache_extend(cache, _dev(seqs), _dev(add))) == m.extend(seqs, add)
    assert cache.lens[torch.tensor(seqs, device="cuda")].tolist() == add
    for bad in ([5, 199999, 5], [7, 200000]):
        bn.bitnet_cache_free(cache, _dev(bad))
        assert cache.errors() == bn.CACHE_ERR_SEQ
    bn.bitnet_cache_fork(cache, _dev([5, 5]), _dev([6, 199998]))
    m.fork([5, 5], [6, 199998])
    bn.bitnet_cache_free(cache, _dev([199999, 5]))
    m.free([199999, 5])
    assert ref.pairs(bn.bitnet_cache_compact(cache)) == m.compact()
    assert cache.refs.tolist() == m.refs and cache.lens.tolist() == m.lens
    for s in (6, 199998, 131071):
        assert cache.table[s].tolist()[:m.pages(m.lens[s])] == m.table[s][:m.pages(m.lens[s])]
    assert cache.errors() == 0


def test_upkeep_workspace_contents_do_not_matter(bn):
    """The same life with scratch of exactly the size asked for, full of ones."""
    for fill in (0, 255):
        cache, m = _make(bn, 70, 9, 40, 8, kv=1)
        n = 6
        size = cache.workspace_size(n)
        buf = torch.full((size + 64,), fill, dtype=torch.uint8, device="cuda")
        ws = buf[:size]

        def again():
            buf.fill_(fill)
            return ws

        bn.bitnet_cache_extend(cache, _dev([0, 1]), _dev([100, 61]), workspace=again())
        m.extend([0, 1], [100, 61])
        bn.bitnet_cache_fork(cache, _dev([0, 1, 1, 0]), _dev([2, 3, 4, 5]), workspace=again())
        m.fork([0, 1, 1, 0], [2, 3, 4, 5])
        seqs, add = [5, 4, 3, 2, 1, 0], [1, 1, 2, 3, 1, 9]
        got = bn.bitnet_cache_extend(cache, _dev(seqs), _dev(add), workspace=again())
        assert ref.pairs(got) == m.extend(seqs, add)
        bn.bitnet_cache_free(cache, _dev([0, 3]), workspace=again())
        m.free([0, 3])
        assert ref.pairs(bn.bitnet_cache_compact(cache, workspace=again())) == m.compact()
        m.check(cache)
        assert torch.all(buf[size:] == fill) and cache.errors() == 0


def test_long_rows(bn):
    """Slots of many pages: forks, frees and compactions over several chunks of a row."""
    cache, m = _make(bn, 9000, 6, 3000, 8, kv=1)
    bn.bitnet_cache_extend(cache, _dev([1, 4]), _dev([20000, 7]))
    m.extend([1, 4], [20000, 7])
    bn.bitnet_cache_fork(cache, _dev([1, 1]), _dev([0, 5]))
    m.fork([1, 1], [0, 5])
    got = bn.bitnet_cache_extend(cache, _dev([0, 4, 5]), _dev([4000, 20000, 1]))
    assert ref.pairs(got) == m.extend([0, 4, 5], [4000, 20000, 1])
    bn.bitnet_cache_free(cache, _dev([1, 5]))
    m.free([1, 5])
    bn.bitnet_cache_free(cache, _dev([0]))
    m.free([0])
    m.check(cache)
    assert ref.pairs(bn.bitnet_cache_compact(cache)) == m.compact()
    m.check(cache)
    assert cache.errors() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("what", ["append", "attention", "copy", "extend", "fork", "free", "compact"])
def test_a_dropped_cache_lives_until_the_given_stream_is_done(bn, what, dtype):
    """A cache that is dropped behind a call on a side stream that has yet to run it: none of its
    memory is handed out before, neither its pools nor its tables, so the call neither reads nor writes
    what others put there."""
    side = torch.cuda.Stream()
    kv, D = 2, 64
    x = torch.ones(2, kv, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, kv, D, dtype=torch.bfloat16, device="cuda")
    slots, one, more = _dev([0, 1]), _dev([1, 1]), _dev([2, 3])
    copies = _dev([1, 0, 0, 9])
    calls = {
        "append": lambda c: bn.bitnet_cache_append(c, 1, x, x, slots, stream=side),
        "attention": lambda c: bn.bitnet_paged_attention(q, c, 1, slots, stream=side),
        "copy": lambda c: bn.bitnet_cache_copy(c, copies, stream=side),
        "extend": lambda c: bn.bitnet_cache_extend(c, slots, one, stream=side),
        "fork": lambda c: bn.bitnet_cache_fork(c, slots, more, stream=side),
        "free": lambda c: bn.bitnet_cache_free(c, slots, stream=side),
        "compact": lambda c: bn.bitnet_cache_compact(c, stream=side),
    }

    def new():
        return bn.make_cache(20, 4, 3, kv, D, 16, 2, dtype)

    seen = 0
    for cycles in (20_000_000, 40_000_000, 400_000_000, 800_000_000):
        cache = new()
        bn.bitnet_cache_extend(cache, slots, _dev([20, 5]))
        bn.bitnet_cache_append(cache, 1, x, x, slots)
        want = bn.bitnet_paged_attention(q, cache, 1, slots)
        mine = cache.layers + [(cache.table, cache.lens, cache.refs, cache.error)]
        mine = {t.data_ptr(): t.numel() * t.element_size() for ts in mine for t in ts}
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(cycles)
        got = calls[what](cache)
        del cache
        others = [new() for _ in range(2)]
        theirs = [t for c in others for ts in c.layers + [(c.table, c.lens, c.refs, c.error)]
                  for t in ts]
        if side.query():  # the host was slower than that: longer
            del others, theirs
            continue
        seen += 1
        for t in theirs:
            at, size = t.data_ptr(), t.numel() * t.element_size()
            assert all(at + size <= p or p + n <= at for p, n in mine.items())
        before = [t.clone() for t in theirs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(theirs, before))
        if what == "attention":
            assert torch.equal(got, want)
        del others, theirs, before, got
        if seen == 2:
            break
    assert seen


def test_errors_waits_for_every_stream(bn):
    """What a call on another stream reports is there as soon as the call has been made: one that named
    the stream, one that ran under it, a replayed graph; and it is cleared before later calls set it."""
    cache, _ = _make(bn, 8, 3, 2, 16)
    side, bad = torch.cuda.Stream(), _dev([1, 1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        bn.bitnet_cache_free(cache, bad)

    def under():
        with torch.cuda.stream(side):
            bn.bitnet_cache_free(cache, bad)

    def replayed():
        with torch.cuda.stream(side):
            graph.replay()

    bn.bitnet_cache_free(cache, bad, stream=side)
    assert cache.errors() == bn.CACHE_ERR_SEQ
    for call in (lambda: bn.bitnet_cache_free(cache, bad, stream=side), under, replayed):
        for _ in range(3):
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
            call()
            assert cache.errors() == bn.CACHE_ERR_SEQ
            call()  # at once behind the clearing
            assert cache.errors() == bn.CACHE_ERR_SEQ and cache.errors() == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("w", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_inf_and_nan_show_in_8_bits(bn, D, w, value):
    """One Inf or NaN in K or V of one token and head: that row's scale is NaN, every other row is as
    without it, and attention gives NaN for the query heads that see it, and what it gave for the
    others."""
    g = np.random.default_rng([D, w])
    x = [ref.bf16(g.standard_normal((30, 3, D))).cuda() for _ in range(2)]
    seqs, pos = _dev([0] * 17 + [1] * 13), _dev(list(range(17)) + list(range(13)))
    q = ref.bf16(g.standard_normal((2, 6, D))).cuda()
    got = []
    for bad in (False, True):
        cache, _ = _make(bn, 8, 2, 4, 16, dtype=torch.int8, kv=3, D=D)
        bn.bitnet_cache_extend(cache, _dev([0, 1]), _dev([17, 13]))
        if bad:
            x[w][20, 1, D - 9] = value  # position 3 of slot 1
        bn.bitnet_cache_append(cache, 0, *x, seqs, pos)
        got.append((cache.layers[0], bn.bitnet_paged_attention(q, cache, return_lse=True)))
        page = int(cache.table[1, 0])
        assert cache.errors() == 0
    (clean, (o, l)), (layer, (ob, lb)) = got
    assert torch.isnan(layer[2 + w][page, 1, 3])
    layer[2 + w][page, 1, 3], layer[w][page, 1, 3] = clean[2 + w][page, 1, 3], clean[w][page, 1, 3]
    assert all(torch.equal(a, b) for a, b in zip(layer, clean))
    assert ob[1, 2:4].isnan().all() and bool(lb[1, 2:4].isnan().all()) == (w == 0)
    ob[1, 2:4], lb[1, 2:4] = o[1, 2:4], l[1, 2:4]
    assert torch.equal(ob, o) and torch.equal(lb, l)
