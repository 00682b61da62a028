"""4-bit weights with group scales (bitnet_pack_w4, bitnet_linear_w4) against plain 64-bit
products. Tolerance: each of the K terms' sums may be off by one binary32 step of the sum of
|terms| (K of them, plus the scale's product), then one rounding to the output type."""
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


def _case(M, N, K, group, seed):
    g = np.random.default_rng([seed, M, N, K, group])
    t = g.integers(-8, 8, (N, K))
    scales = ref.bf16(g.uniform(1e-3, 2e-2, (N, -(-K // group))))
    return ref.bf16(g.standard_normal((M, K))), t, scales


def _check(y, x, t, scales, group, where=""):
    want, size = ref.w4_linear(x, t, scales, group)
    tol = (x.shape[1] + 2) * ref.F32_STEP * size + 1e-30
    if y.dtype == torch.bfloat16:
        tol = tol + ref.BF16_HALF * (np.abs(want) + tol)
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"{where}: {np.max(err / tol):.2f} of the tolerance"


@pytest.mark.parametrize("N,K,group", [(1, 64, 32), (17, 192, 128), (40, 2560, 128),
                                       (129, 6912, 64), (16, 14336, 32)])
def test_pack_matches_the_format(bn, N, K, group):
    W = np.random.default_rng([K, N]).standard_normal((N, K)).astype(np.float32)
    W[0, :32] = 0.0  # a group of zeros takes the smallest scale
    W[N - 1, K - 1] = 40.0
    packed, scales = bn.bitnet_pack_w4(torch.from_numpy(W).cuda(), group)
    t, s = ref.w4_quantise(W, group)
    assert torch.equal(scales.cpu().view(torch.int16), s.view(torch.int16))
    assert np.array_equal(packed.cpu().numpy(), ref.w4_pack_codes(t))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 1, 64), (1, 640, 2560), (1, 33, 192), (2, 130, 6912),
                                   (3, 2047, 320), (8, 257, 4096), (9, 31, 1088), (16, 96, 128),
                                   (33, 100, 2560), (1, 47, 14336), (70, 19, 704)])
def test_linear(bn, M, N, K, group, out):
    x, t, scales = _case(M, N, K, group, 1)
    packed = torch.from_numpy(ref.w4_pack_codes(t)).cuda()
    y = bn.bitnet_linear_w4(x.cuda(), packed, scales.cuda(), group, out_dtype=out)
    assert y.shape == (M, N) and y.dtype == out
    _check(y, x, t, scales, group, f"{M}x{N}x{K} g{group}")
    again = bn.bitnet_linear_w4(x.cuda(), packed, scales.cuda(), group, out_dtype=out)
    assert torch.equal(y, again)


def test_linear_more_rows_than_one_wave(bn):
    """More weight rows than the GPU holds at once, and an odd number of them."""
    x, t, scales = _case(2, 20011, 256, 64, 2)
    y = bn.bitnet_linear_w4(x.cuda(), torch.from_numpy(ref.w4_pack_codes(t)).cuda(), scales.cuda(),
                            64, out_dtype=torch.float32)
    _check(y, x, t, scales, 64)


@pytest.mark.parametrize("M,K,group", [(5, 64 * 1031, 128), (2, 32768, 32), (1, 65536, 64),
                                       (17, 32704, 32), (9, 32768, 32), (40, 131072, 128)])
def test_linear_long_rows(bn, M, K, group):
    """Up to the longest rows; x past what shared memory holds."""
    x, t, scales = _case(M, 24, K, group, 3)
    y = bn.bitnet_linear_w4(x.cuda(), torch.from_numpy(ref.w4_pack_codes(t)).cuda(), scales.cuda(),
                            group, out_dtype=torch.float32)
    _check(y, x, t, scales, group)


def test_rows_of_x_do_not_meet(bn):
    """An Inf or NaN in one token leaves the other tokens' outputs as they are."""
    x, t, scales = _case(5, 64, 512, 64, 4)
    packed, sc = torch.from_numpy(ref.w4_pack_codes(t)).cuda(), scales.cuda()
    y = bn.bitnet_linear_w4(x.cuda(), packed, sc, 64)
    x[2, 7], x[2, 300] = float("inf"), float("nan")
    z = bn.bitnet_linear_w4(x.cuda(), packed, sc, 64)
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], z[keep])


def test_extreme_codes_and_scales(bn):
    """All codes at their ends, and scales from 2^-100 to 2^100."""
    x, t, _ = _case(1, 32, 256, 128, 5)
    t[:] = np.where(np.arange(256) % 2, 7, -8)
    scales = ref.bf16(2.0 ** np.linspace(-100, 100, 64).reshape(32, 2))
    y = bn.bitnet_linear_w4(x.cuda(), torch.from_numpy(ref.w4_pack_codes(t)).cuda(), scales.cuda(),
                            128, out_dtype=torch.float32)
    _check(y, x, t, scales, 128)


def test_output_is_written_whole_and_nothing_else(bn):
    """y sits in a larger buffer whose other bytes stay."""
    x, t, scales = _case(3, 37, 320, 32, 6)
    buf = torch.full((3 * 37 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:111].view(3, 37)
    bn.bitnet_linear_w4(x.cuda(), torch.from_numpy(ref.w4_pack_codes(t)).cuda(), scales.cuda(), 32,
                        y=y)
    _check(y, x, t, scales, 32)
    assert torch.all(buf[111:] == 7.0)


def test_streams_and_graph(bn):
    """On a side stream, and captured and replayed with new inputs."""
    x, t, scales = _case(4, 200, 1024, 64, 7)
    packed, sc, xd = torch.from_numpy(ref.w4_pack_codes(t)).cuda(), scales.cuda(), x.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = bn.bitnet_linear_w4(xd, packed, sc, 64, stream=side)
    side.synchronize()
    _check(y, x, t, scales, 64)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        yg = bn.bitnet_linear_w4(xd, packed, sc, 64)
    x2 = ref.bf16(np.random.default_rng(8).standard_normal((4, 1024)))
    xd.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    _check(yg, x2, t, scales, 64)


def _large(N, K, group, seed):
    """Random packed weights, their values and scales, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = -(-K // 128)
    packed = torch.randint(0, 256, (N, blocks * 64), generator=g, device="cuda",
                           dtype=torch.int32).to(torch.uint8)
    words = packed.view(torch.int32).view(N, blocks, 4, 4)  # c, j
    t = torch.stack([(words >> (2 * i + 14 if i & 1 else 2 * i) & 15) - 8 for i in range(8)], -1)
    t = t.permute(0, 1, 3, 2, 4).reshape(N, blocks * 128)[:, :K]
    if K % 128:  # weights past K have code 8
        half = words[:, -1, :, 2:]
        half.fill_(-0x77777778)
    scales = torch.rand(N, -(-K // group), generator=g, device="cuda") * 0.02 + 0.001
    return packed, t, scales.to(torch.bfloat16)


def _check_large(y, x, t, scales, group):
    """As _check, and every value of x may be off by 2^-29 of the largest of its block of 128: it is
    taken in units of 2^-28 times the power of two below that, rounded once. (Sums of hundreds of
    values at the end of binary32's range are off by a step of 2^-149 each at most.)"""
    K = t.shape[1]
    w = t.double() * scales.double().repeat_interleave(group, 1)[:, :K]
    xd = x.double()
    want, size = xd @ w.T, xd.abs() @ w.abs().T
    pad = torch.nn.functional.pad(xd.abs(), (0, -K % 128)).view(x.shape[0], -1, 128)
    off = (pad.amax(2, keepdim=True) * 2.0 ** -29).expand_as(pad).reshape(x.shape[0], -1)[:, :K]
    tol = (K + 2) * ref.F32_STEP * size + off @ w.abs().T + 2.0 ** -140
    if y.dtype == torch.bfloat16:
        tol = tol + ref.BF16_HALF * (want.abs() + tol)
    err = (y.double() - want).abs()
    assert torch.all(err <= tol), f"{(err / tol).max().item():.2f} of the tolerance"


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,group", [(1, 2560, 6912, 128), (1, 8001, 2112, 64),
                                         (1, 601, 28160, 32), (2, 17001, 1984, 128),
                                         (2, 14336, 2560, 32), (2, 700, 48000, 64),
                                         (3, 35001, 1984, 128), (4, 28672, 2560, 128),
                                         (4, 1600, 42048, 128), (4, 28672, 2560, 64),
                                         (1, 9601, 192, 32), (5, 10007, 2048, 32),
                                         (8, 9999, 4160, 128), (2, 9473, 8192, 128),
                                         (7, 9500, 8192, 128), (1, 40000, 64, 64),
                                         (8, 14336, 4096, 64), (3, 10240, 4096, 32),
                                         (9, 9601, 2112, 64), (33, 9480, 1088, 32)])
def test_large_layers_at_few_tokens(bn, M, N, K, group, out):
    packed, t, scales = _large(N, K, group, N)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    y = bn.bitnet_linear_w4(x, packed, scales, group, out_dtype=out)
    _check_large(y, x, t, scales, group)
    assert torch.equal(y, bn.bitnet_linear_w4(x, packed, scales, group, out_dtype=out))


@pytest.mark.parametrize("M", [1, 2, 4])
def test_large_layers_wide_ranges_of_x(bn, M):
    """Values of one row from 2^-130 to 2^100: outliers in their blocks, blocks of zeros, of the
    type's largest and smallest values, of one magnitude each, all ones and all signs."""
    N, K = 28672, 2560
    packed, t, scales = _large(N, K, 128, 9)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, 3] = 3e4
    x[:, 128:256] *= 2.0 ** -torch.randint(0, 40, (M, 128), generator=g, device="cuda")
    x[:, 256:384] = 0.0
    x[:, 384:512] *= 1e-37
    x[:, 512:640] = 2.0 ** -130
    x[:, 640:768] = 1.9921875  # all bits of the mantissa
    x[:, 768:896] = -1.9921875
    x[:, 900] = 1.0 / 3
    x = x.to(torch.bfloat16)
    for rows in (x, x * 2.0 ** 60, x * 2.0 ** 110, x * 2.0 ** -100):
        y = bn.bitnet_linear_w4(rows, packed, scales, 128, out_dtype=torch.float32)
        _check_large(y, rows, t, scales, 128)
    tiny = torch.full((M, K), 2.0 ** -126, dtype=torch.bfloat16, device="cuda")
    y = bn.bitnet_linear_w4(tiny, packed, torch.full_like(scales, 1024.0), 128,
                            out_dtype=torch.float32)
    _check_large(y, tiny, t, torch.full_like(scales, 1024.0), 128)
    ends = (packed & 0) + 0x0F  # codes 15 and 0: 7 and -8
    te = torch.where(((ends.view(torch.int32).view(N, -1, 4, 4)[..., None] >> torch.tensor(
        [2 * i + 14 if i & 1 else 2 * i for i in range(8)], device="cuda")) & 15) == 15, 7, -8)
    te = te.permute(0, 1, 3, 2, 4).reshape(N, K)
    big = torch.full((M, K), 2.0 ** 64 * 1.9921875, dtype=torch.bfloat16, device="cuda")
    for sign in (1, -1):
        y = bn.bitnet_linear_w4(big * sign, ends, scales, 128, out_dtype=torch.float32)
        _check_large(y, big * sign, te, scales, 128)


def test_large_layers_nan_stays_in_its_row(bn):
    N, K = 28672, 2560
    packed, t, scales = _large(N, K, 128, 10)
    g = torch.Generator(device="cuda").manual_seed(1)
    for M in (2, 4):
        x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
        y = bn.bitnet_linear_w4(x, packed, scales, 128)
        for value in (float("nan"), float("inf")):
            bad = x.clone()
            bad[1, 777] = value
            z = bn.bitnet_linear_w4(bad, packed, scales, 128)
            assert z[1].isnan().all()
            keep = [m for m in range(M) if m != 1]
            assert torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("M,N,K,group", [(1, 640, 2560, 128), (2, 2560, 6912, 64),
                                         (8, 10000, 1024, 32), (3, 96, 32768, 32)])
def test_packed_anew_and_used_at_once(bn, M, N, K, group):
    """Weights packed into the buffers that the calls before have read, and multiplied by the next call
    of the stream: the results are those of weights that were there long before."""
    g = torch.Generator(device="cuda").manual_seed(N)
    Ws = [torch.randn(N, K, generator=g, device="cuda") * 2.0 ** i for i in range(3)]
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    want = []
    for W in Ws:
        packed, scales = bn.bitnet_pack_w4(W, group)
        torch.cuda.synchronize()
        want.append(bn.bitnet_linear_w4(x, packed, scales, group, out_dtype=torch.float32))
    stream = torch.cuda.current_stream().cuda_stream
    got = []
    for i in range(30):
        assert bn.lib.bitnet_pack_w4(Ws[i % 3].data_ptr(), N, K, group, packed.data_ptr(),
                                     scales.data_ptr(), stream) == bn.OK
        got.append([bn.bitnet_linear_w4(x, packed, scales, group, out_dtype=torch.float32)
                    for _ in range(2)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 3]) for i, ys in enumerate(got) for y in ys)


@pytest.mark.parametrize("far", [4, 8, 14, 20, 26])
@pytest.mark.parametrize("M,N,K,group", [(1, 28672, 2560, 128), (1, 6912, 2560, 32),
                                         (2, 14336, 4096, 64), (3, 28672, 2560, 128),
                                         (4, 131071, 576, 128)])
def test_large_layers_low_digits(bn, M, N, K, group, far):
    """The small values of a block are the whole result: its largest, 2^far times as large, meets codes
    of t = 0. Up to 2^20 no bit of x is cut off, beyond it is off by 2^-29 of the largest of its block.
    Sums within a group are exact, so beside that there is a binary32 step for each group, of sums
    whose digits are up to four times the terms, and some for joining digits and warps."""
    packed, t, scales = _large(N, K, group, 11)
    at = torch.arange(0, K, 128, device="cuda") + 37  # one value of each block
    words = packed.view(torch.int32).view(N, -1, 16)
    # weight 37 = 32 * 1 + 8 * 0 + 5: word 1, bits 24 to 27
    words[:, :, 1] = (words[:, :, 1] & ~(15 << 24)) | 8 << 24
    t = t.clone()
    t[:, at] = 0
    g = torch.Generator(device="cuda").manual_seed(M)
    small = torch.rand(M, K, generator=g, device="cuda") + 1
    small *= torch.randint(0, 2, (M, K), generator=g, device="cuda") * 2 - 1
    x = small * 2.0 ** -far
    x[:, at] = 1.9921875 * (torch.randint(0, 2, (M, len(at)), generator=g, device="cuda") * 2 - 1)
    x = x.to(torch.bfloat16)
    w = t.double() * scales.double().repeat_interleave(group, 1)[:, :K]
    xd = x.double()
    want, size = xd @ w.T, xd.abs() @ w.abs().T
    tol = 4 * (scales.shape[1] + 20) * ref.F32_STEP * size
    if far > 20:
        tol = tol + 2.0 ** -29 * 1.9921875 * w.abs().sum(1)
    y = bn.bitnet_linear_w4(x, packed, scales, group, out_dtype=torch.float32)
    err = (y.double() - want).abs()
    assert torch.all(err <= tol), f"{(err / tol).max().item():.2f} of the tolerance"
    # to the bit where nothing of x is cut off: one block, one group, one value
    if group == 128:
        x.zero_()
        x[:, 37] = -1.9921875
        x[:, 100] = 1.9921875 * 2.0 ** -21
        y = bn.bitnet_linear_w4(x, packed, scales, group, out_dtype=torch.float32)
        assert torch.equal(y, (x[:, 100:101].double() @ w[:, 100:101].T).float())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,group", [(17, 14336, 4096, 128), (35, 14336, 4096, 32),
                                         (17, 2560, 16384, 64), (35, 2560, 16384, 128),
                                         (100, 4736, 8192, 32), (33, 600, 60032, 64)])
def test_large_layers_several_token_tiles(bn, M, N, K, group, out):
    """More than 16 tokens of layers of more than 2^25 weights: passes of 16, the last cut; teams of four
    and of eight; x through shared memory and L1."""
    packed, t, scales = _large(N, K, group, N)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    y = bn.bitnet_linear_w4(x, packed, scales, group, out_dtype=out)
    w = t.double() * scales.double().repeat_interleave(group, 1)[:, :K]
    want, size = x.double() @ w.T, x.double().abs() @ w.abs().T
    tol = (K + 2) * ref.F32_STEP * size
    if out == torch.bfloat16:
        tol = tol + ref.BF16_HALF * (want.abs() + tol)
    err = (y.double() - want).abs()
    assert torch.all(err <= tol), f"{(err / tol).max().item():.2f} of the tolerance"


def test_more_tokens_than_one_launch(bn):
    """65535 * 16 + 3 tokens: rows on both sides of the split, and nothing behind the last."""
    M, N, K = 65535 * 16 + 3, 5, 64
    packed, t, scales = _large(N, K, 64, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    buf = torch.full((M * N + 64,), 7.0, device="cuda")
    y = bn.bitnet_linear_w4(x, packed, scales, 64, y=buf[:M * N].view(M, N))
    w = t.double() * scales.double().repeat_interleave(64, 1)[:, :K]
    want, size = x.double() @ w.T, x.double().abs() @ w.abs().T
    assert torch.all((y.double() - want).abs() <= (K + 2) * ref.F32_STEP * size)
    assert torch.all(buf[M * N:] == 7.0)
