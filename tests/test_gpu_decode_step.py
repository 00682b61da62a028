"""A decode step as a user runs it: q/k/v from one bitnet_linear_batch, the cache grown and
written, attention, the output projection from bitnet_linear and a 4-bit output table, over two
layers, for beams that fork, with the whole step captured into one CUDA graph."""
import numpy as np
import pytest
import torch

import decode_ref as ref
import synth

pytestmark = pytest.mark.gpu

K, HEADS, KV, D, PAGE, VOCAB, LAYERS = 256, 4, 2, 64, 16, 301, 2


@pytest.fixture(scope="module")
def bn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ternary_w2a8_linear_token_b200 as bn
    return bn


def _dev(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """Weights, cache and one step over all slots of `seqs`."""

    def __init__(self, bn, dtype, B):
        self.bn, self.B = bn, B
        g = synth.rng(0, 11, 3, 0, synth.KIND_T)

        def ternary(N):
            t = torch.from_numpy(synth.ternary(N, K, g, 0.4)).cuda()
            return bn.bitnet_pack_ternary(t), torch.from_numpy(synth.uniform_scale(1, g)).cuda() / 16

        self.layers = []
        for _ in range(LAYERS):
            qkv = [ternary(n) + (False,) for n in (HEADS * D, KV * D, KV * D)]
            self.layers.append((qkv, ternary(K)))
        W = torch.from_numpy(g.standard_normal((VOCAB, K)).astype(np.float32)).cuda()
        self.table4, self.scales4 = bn.bitnet_pack_w4(W, 64)
        self.cache = bn.make_cache(200, 8, 12, KV, D, PAGE, LAYERS, dtype)
        self.model = ref.Model(200, 8, 12, PAGE)
        self.x = torch.zeros(B, K, dtype=torch.bfloat16, device="cuda")
        self.seqs = _dev(list(range(B)))
        self.add = _dev([1] * B)

    def run(self):
        bn, seen = self.bn, []
        copies = bn.bitnet_cache_extend(self.cache, self.seqs, self.add)
        bn.bitnet_cache_copy(self.cache, copies)
        h = self.x
        for i, (qkv, o) in enumerate(self.layers):
            q, k, v = bn.bitnet_linear_batch(h, qkv)
            bn.bitnet_cache_append(self.cache, i, k, v, seqs=self.seqs)
            a, lse = bn.bitnet_paged_attention(q, self.cache, i, seqs=self.seqs, return_lse=True)
            seen.append((q, k, v, a, lse))
            h = bn.bitnet_linear(a, *o, False)
        return seen, h, bn.bitnet_linear_w4(h, self.table4, self.scales4, 64,
                                            out_dtype=torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_captured_decode_with_forks(bn, dtype):
    B = 6
    st = Step(bn, dtype, B)
    cache, m = st.cache, st.model
    # a prompt of 21 tokens in slot 0, forked into the other beams
    g = torch.Generator(device="cuda").manual_seed(5)
    bn.bitnet_cache_extend(cache, _dev([0]), _dev([21]))
    m.extend([0], [21])
    held = [[[] for _ in range(8)] for _ in range(LAYERS)]  # what each slot should hold
    for i in range(LAYERS):
        k, v = (torch.randn(21, KV, D, generator=g, device="cuda").to(torch.bfloat16)
                for _ in range(2))
        bn.bitnet_cache_append(cache, i, k, v, seqs=_dev([0] * 21), pos=_dev(list(range(21))))
        held[i][0] = [(k[t], v[t]) for t in range(21)]
    bn.bitnet_cache_fork(cache, _dev([0] * 5), _dev([1, 2, 3, 4, 5]))
    m.fork([0] * 5, [1, 2, 3, 4, 5])
    for i in range(LAYERS):
        for s in range(1, 6):
            held[i][s] = list(held[i][0])
    start = cache.table.clone(), cache.lens.clone(), cache.refs.clone()
    st.x.copy_(torch.randn(B, K, generator=g, device="cuda"))
    st.run()  # eagerly once, then back to the start
    for t, s in zip((cache.table, cache.lens, cache.refs), start):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        seen, h, logits = st.run()
    for step in range(25):
        st.x.copy_(torch.randn(B, K, generator=g, device="cuda"))
        if step == 9:  # beam 2 is dropped and takes beam 4's place; the pool is compacted
            bn.bitnet_cache_free(cache, _dev([2]))
            bn.bitnet_cache_fork(cache, _dev([4]), _dev([2]))
            moves = bn.bitnet_cache_compact(cache)
            bn.bitnet_cache_copy(cache, moves)
            m.free([2])
            m.fork([4], [2])
            assert ref.pairs(moves) == m.compact()
            for i in range(LAYERS):
                held[i][2] = list(held[i][4])
        graph.replay()
        torch.cuda.synchronize()
        m.extend(list(range(B)), [1] * B)
        m.check(cache)
        for i, (q, k, v, a, lse) in enumerate(seen):
            for b in range(B):
                held[i][b].append((k[b].view(KV, D).clone(), v[b].view(KV, D).clone()))
            if step in (0, 8, 9, 10, 24):
                for b in range(B):
                    kv = []
                    for w in range(2):
                        x = torch.stack([tok[w] for tok in held[i][b]]).cpu()
                        if dtype == torch.int8:
                            qq, s = ref.quantise(x)
                            kv.append(qq.astype(np.float64) / s.astype(np.float64)[..., None])
                        else:
                            kv.append(x.double().numpy())
                    o, l, to, tl = ref.attention(q[b].view(HEADS, D).double().cpu().numpy(), *kv,
                                                 D ** -0.5)
                    err = np.abs(a[b].view(HEADS, D).double().cpu().numpy() - o)
                    assert np.all(err <= to + ref.BF16_HALF * (np.abs(o) + to)), (step, i, b)
                    assert np.all(np.abs(lse[b].double().cpu().numpy() - l) <= tl)
        assert torch.equal(h, bn.bitnet_linear(seen[-1][3], *st.layers[-1][1], False))
        assert torch.equal(logits, bn.bitnet_linear_w4(h, st.table4, st.scales4, 64,
                                                       out_dtype=torch.float32))
    assert cache.errors() == 0 and bn.bitnet_check_device_errors() == 0
