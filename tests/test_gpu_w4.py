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
