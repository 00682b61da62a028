"""Host-side refusals of the decode-step calls: every call here fails its argument checks, which
run before the library touches CUDA (fake pointers are never dereferenced)."""
import ctypes
import re
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def bn():
    import ternary_w2a8_linear_token_b200 as bn
    return bn


def test_structs_and_constants_match_the_header(bn):
    assert ctypes.sizeof(bn.bitnet_cache) == 72 and bn.bitnet_cache.page_size.offset == 56
    assert ctypes.sizeof(bn.bitnet_cache_layer) == 32
    src = open(os.path.join(ROOT, "include", "bitnet.h"), encoding="utf-8").read()
    for name, shift in re.findall(r"#define BITNET_(CACHE_ERR_[A-Z]+) \(1 << (\d+)\)", src):
        assert getattr(bn, name) == 1 << int(shift)
    assert f"BITNET_CACHE_MAX_LAYERS {bn.CACHE_MAX_LAYERS}" in src


def test_w4_refusals(bn):
    L = bn.lib
    assert [L.bitnet_w4_row_bytes(k) for k in (-1, 0, 1, 64, 128, 192, 6912)] == \
        [0, 0, 64, 64, 64, 128, 3456]

    def pack(W=FAKE, N=4, K=128, group=64, p=FAKE, s=FAKE):
        return L.bitnet_pack_w4(W, N, K, group, p, s, None)

    def lin(x=FAKE, M=1, K=128, p=FAKE, s=FAKE, group=64, N=4, y=FAKE, od=0):
        return L.bitnet_linear_w4(x, M, K, p, s, group, N, y, od, None)

    for kw in (dict(W=None), dict(p=None), dict(s=None)):
        assert pack(**kw) == bn.ERR_NULL
    for kw in (dict(x=None), dict(p=None), dict(s=None), dict(y=None)):
        assert lin(**kw) == bn.ERR_NULL
    for f in (pack, lin):
        assert f(K=0) == f(K=66) == f(N=0) == f(N=1 << 31) == bn.ERR_SHAPE
        assert f(K=96) == f(group=16) == f(group=256) == f(group=0) == bn.ERR_UNSUPPORTED
        assert f(p=FAKE + 8) == f(s=FAKE + 1) == bn.ERR_ALIGN
    assert pack(W=FAKE + 4) == lin(x=FAKE + 2) == lin(y=FAKE + 4) == bn.ERR_ALIGN
    assert lin(M=0) == lin(M=1 << 31) == bn.ERR_SHAPE
    assert lin(od=2) == lin(od=-1) == bn.ERR_UNSUPPORTED
    assert lin(K=64 * 1024 + 64) == lin(K=32 * 1024 + 64, group=32) == bn.ERR_UNSUPPORTED


def _cache(bn, **kw):
    f = dict(table=FAKE, lens=FAKE, refs=FAKE, error=FAKE, num_pages=100, max_seqs=8, max_pages=16,
             page_size=16, kv_heads=2, head_dim=128, dtype=0)
    f.update(kw)
    return bn.bitnet_cache(**f)


def _calls(bn):
    """Every cache call with arguments that pass all checks but those of the descriptor."""
    L, big = bn.lib, 1 << 40
    lay = (bn.bitnet_cache_layer * 1)(bn.bitnet_cache_layer(FAKE, FAKE, FAKE, FAKE))
    return {
        "fork": lambda c: L.bitnet_cache_fork(c, FAKE, FAKE, 1, FAKE, big, None),
        "extend": lambda c: L.bitnet_cache_extend(c, FAKE, FAKE, 1, FAKE, 1, FAKE, big, None),
        "free": lambda c: L.bitnet_cache_free(c, FAKE, 1, FAKE, big, None),
        "compact": lambda c: L.bitnet_cache_compact(c, FAKE, 1 << 30, FAKE, big, None),
        "copy": lambda c: L.bitnet_cache_copy(c, lay, 1, FAKE, 1, None),
        "append": lambda c: L.bitnet_cache_append(c, lay, FAKE, FAKE, 1, None, None, None),
        "attention": lambda c: L.bitnet_paged_attention(c, lay, FAKE, 1, c.kv_heads, None, 1.0, 0,
                                                        0, FAKE, None, FAKE, big, None),
    }


@pytest.mark.parametrize("name", ["fork", "extend", "free", "compact", "copy", "append",
                                  "attention"])
def test_descriptor_refusals(bn, name):
    call = _calls(bn)[name]
    for kw in (dict(table=None), dict(lens=None), dict(refs=None), dict(error=None)):
        assert call(_cache(bn, **kw)) == bn.ERR_NULL
    for kw in (dict(num_pages=0), dict(num_pages=(1 << 30) + 1), dict(max_seqs=0),
               dict(max_seqs=(1 << 24) + 1), dict(max_pages=0), dict(max_pages=(1 << 26) + 1),
              
               dict(kv_heads=0), dict(kv_heads=1025)):
        assert call(_cache(bn, **kw)) == bn.ERR_SHAPE, kw
    for kw in (dict(page_size=0), dict(page_size=4), dict(page_size=24), dict(page_size=512),
               dict(head_dim=32), dict(head_dim=96), dict(head_dim=256), dict(dtype=2),
               dict(num_pages=1 << 27)):
        assert call(_cache(bn, **kw)) == bn.ERR_UNSUPPORTED, kw
    for kw in (dict(table=FAKE + 2), dict(lens=FAKE + 1), dict(refs=FAKE + 2),
               dict(error=FAKE + 2)):
        assert call(_cache(bn, **kw)) == bn.ERR_ALIGN


def test_upkeep_refusals(bn):
    L, c, big = bn.lib, _cache(bn), 1 << 40
    n = 1 << 24
    assert L.bitnet_cache_fork(c, None, FAKE, 1, FAKE, big, None) == bn.ERR_NULL
    assert L.bitnet_cache_fork(c, FAKE, None, 1, FAKE, big, None) == bn.ERR_NULL
    assert L.bitnet_cache_fork(c, FAKE, FAKE, 0, FAKE, big, None) == bn.ERR_SHAPE
    assert L.bitnet_cache_fork(c, FAKE, FAKE, n + 1, FAKE, big, None) == bn.ERR_SHAPE
    assert L.bitnet_cache_fork(c, FAKE, FAKE + 2, 1, FAKE, big, None) == bn.ERR_ALIGN
    assert L.bitnet_cache_fork(c, FAKE, FAKE, 1, None, big, None) == bn.ERR_WORKSPACE
    need = L.bitnet_cache_workspace_size(c, 1)
    assert L.bitnet_cache_fork(c, FAKE, FAKE, 1, FAKE, need - 1, None) == bn.ERR_WORKSPACE
    assert L.bitnet_cache_fork(c, FAKE, FAKE, 1, FAKE + 16, big, None) == bn.ERR_ALIGN
    assert L.bitnet_cache_extend(c, FAKE, None, 1, FAKE, 1, FAKE, big, None) == bn.ERR_NULL
    assert L.bitnet_cache_extend(c, FAKE, FAKE, 1, None, 1, FAKE, big, None) == bn.ERR_NULL
    assert L.bitnet_cache_extend(c, FAKE, FAKE, 3, FAKE, 2, FAKE, big, None) == bn.ERR_WORKSPACE
    assert L.bitnet_cache_extend(c, FAKE, FAKE, 1, FAKE + 4, 1, FAKE, big, None) == bn.ERR_ALIGN
    assert L.bitnet_cache_free(c, None, 1, FAKE, big, None) == bn.ERR_NULL
    assert L.bitnet_cache_free(c, FAKE, -1, FAKE, big, None) == bn.ERR_SHAPE
    assert L.bitnet_cache_free(c, FAKE, 1, FAKE, 0, None) == bn.ERR_WORKSPACE
    assert L.bitnet_cache_compact(c, None, 100, FAKE, big, None) == bn.ERR_NULL
    assert L.bitnet_cache_compact(c, FAKE, 49, FAKE, big, None) == bn.ERR_WORKSPACE
    assert L.bitnet_cache_compact(c, FAKE, 50, FAKE, 0, None) == bn.ERR_WORKSPACE
    assert L.bitnet_cache_workspace_size(_cache(bn, kv_heads=0), 1) == 0
    assert L.bitnet_cache_workspace_size(None, 1) == 0
    assert L.bitnet_cache_workspace_size(c, -1) == 0


def test_copy_and_append_refusals(bn):
    L, c = bn.lib, _cache(bn)
    lay = (bn.bitnet_cache_layer * 65)(*[bn.bitnet_cache_layer(FAKE, FAKE, None, None)] * 65)
    assert L.bitnet_cache_copy(c, None, 1, FAKE, 1, None) == bn.ERR_NULL
    assert L.bitnet_cache_copy(c, lay, 1, None, 1, None) == bn.ERR_NULL
    assert L.bitnet_cache_copy(c, lay, 0, FAKE, 1, None) == bn.ERR_SHAPE
    assert L.bitnet_cache_copy(c, lay, 65, FAKE, 1, None) == bn.ERR_SHAPE
    assert L.bitnet_cache_copy(c, lay, 1, FAKE, -1, None) == bn.ERR_SHAPE
    assert L.bitnet_cache_copy(c, lay, 64, FAKE, 0, None) == bn.OK  # nothing to launch
    i8 = _cache(bn, dtype=1)
    assert L.bitnet_cache_copy(i8, lay, 1, FAKE, 1, None) == bn.ERR_NULL  # no scales
    lay[1].v = None
    assert L.bitnet_cache_copy(c, lay, 2, FAKE, 1, None) == bn.ERR_NULL
    lay[1].v = FAKE + 8
    assert L.bitnet_cache_copy(c, lay, 2, FAKE, 1, None) == bn.ERR_ALIGN
    f = L.bitnet_cache_append
    assert f(c, lay, None, FAKE, 1, None, None, None) == bn.ERR_NULL
    assert f(c, None, FAKE, FAKE, 1, None, None, None) == bn.ERR_NULL
    assert f(c, lay, FAKE, FAKE, 0, None, None, None) == bn.ERR_SHAPE
    assert f(c, lay, FAKE, FAKE + 8, 1, None, None, None) == bn.ERR_ALIGN
    assert f(c, lay, FAKE, FAKE, 1, FAKE + 1, None, None) == bn.ERR_ALIGN
    assert f(i8, lay, FAKE, FAKE, 1, None, None, None) == bn.ERR_NULL


def test_attention_refusals(bn):
    c, big = _cache(bn), 1 << 40
    lay = (bn.bitnet_cache_layer * 1)(bn.bitnet_cache_layer(FAKE, FAKE, None, None))

    def call(q=FAKE, B=2, heads=8, seqs=None, scale=1.0, window=0, sinks=0, out=FAKE, lse=None,
             ws=FAKE, wsb=big, layer=lay):
        return bn.lib.bitnet_paged_attention(c, layer, q, B, heads, seqs, scale, window, sinks, out,
                                             lse, ws, wsb, None)

    assert call(q=None) == call(out=None) == call(layer=None) == bn.ERR_NULL
    assert call(B=0) == call(B=(1 << 20) + 1) == call(heads=7) == call(heads=0) == bn.ERR_SHAPE
    assert call(heads=16386) == call(window=-1) == call(sinks=-1) == bn.ERR_SHAPE
    assert call(scale=float("nan")) == call(scale=float("inf")) == bn.ERR_UNSUPPORTED
    assert call(scale=2.5e38) == call(scale=-2.5e38) == bn.ERR_UNSUPPORTED
    assert call(q=FAKE + 8) == call(out=FAKE + 2) == call(lse=FAKE + 2) == bn.ERR_ALIGN
    assert call(seqs=FAKE + 2) == call(ws=FAKE + 128) == bn.ERR_ALIGN
    size = bn.lib.bitnet_paged_attention_workspace_size
    assert call(ws=None) == call(wsb=size(c, 2, 8) - 1) == bn.ERR_WORKSPACE
    assert size(c, 2, 7) == size(c, 0, 8) == size(_cache(bn, page_size=3), 2, 8) == 0


def test_binding_refusals_on_cpu_tensors(bn):
    """The binding refuses tensors that are not on a GPU, and shapes that do not fit."""
    x = torch.zeros(1, 128, dtype=torch.bfloat16)
    packed, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bn.bitnet_linear_w4(x, packed, scales, 64)
    with pytest.raises(ValueError):
        bn.bitnet_linear_w4(x, packed[:, :32], scales, 64)
    with pytest.raises(ValueError):
        bn.bitnet_linear_w4(x, packed, scales, 128)
    with pytest.raises(ValueError):
        bn.bitnet_pack_w4(torch.zeros(4, 128), 64)
    with pytest.raises(ValueError):
        bn.PagedCache(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                      torch.zeros(8, dtype=torch.int32),
                      [(torch.zeros(8, 1, 16, 64, dtype=torch.bfloat16),) * 2])
