"""moe_gemv_nvfp4 at the ends of the activations' range: as long as the terms x * fp4 * e4m3 and their sums are within
fp32's, so is every value on the way, however many pairs name an expert and whatever the scales are.

Tolerances, with u = 2^-24: (K + 3) u sum|terms| as for ordinary values; below 2^-126 a rounding is off by 2^-150
instead, doubled where sums are halved, and K values take at most 2 K roundings: 2 K 2^-149 more. An fp32 output
adds u of the value, a bf16 one 2^-8."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U, B = 2.0 ** -24, 2.0 ** -8
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def weights(P, N, K, scales, seed):
    """Random codes, scale bytes chosen among `scales`, outer scale 1; and their fp64 values."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g)
    sc = torch.tensor(scales)[torch.randint(0, len(scales), (N, K // 16), generator=g)].to(torch.uint8)
    grid = torch.cat([GRID, -GRID])
    v = torch.stack([grid[codes % 16], grid[codes // 16]], 2).flatten(1)
    w = v * sc.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return P.NVFP4(codes.to(torch.uint8).to(DEV), sc.to(DEV), torch.ones(1, device=DEV), N), w.to(DEV)


def check(P, pairs, K, scales, x):
    N = 64
    wq, w = weights(P, N, K, scales, pairs + K)
    y = x.double() @ w.t()
    mag = x.double().abs() @ w.abs().t()
    assert float(mag.max()) < 2.0 ** 127
    e = (K + 3) * U * mag + 2 * K * 2.0 ** -149
    ids = torch.zeros((pairs, 1), dtype=torch.int32, device=DEV)
    ones = torch.ones((pairs, 1), device=DEV)
    for epi, b in ((P.EPI_F32, U), (P.EPI_BF16, B)):
        # half a step of the output's type, below its smallest normal value 2^-134 in bf16
        bound = e + b * 1.02 * y.abs() + (0.0 if epi == P.EPI_F32 else 2.0 ** -134)
        for got in (P.moe_gemv_nvfp4(x, wq, N, epilogue=epi), P.moe_gemv_nvfp4(x, wq, N, ids, epi)[:, 0],
                    P.moe_gemv_nvfp4(x, wq, N, ids, epi, gates=ones)):
            bad = ~((got.double() - y).abs() <= bound)
            assert not bad.any(), f"epilogue {epi}: {int(bad.sum())} values, first {got[bad][0]} for {y[bad][0]}"


def values(pairs, K, low, high, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.rand((pairs, K), generator=g) * (high - low) + low
    return (x * (1 - 2 * torch.randint(0, 2, (pairs, K), generator=g))).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("pairs", [1, 2, 3, 17])
@pytest.mark.parametrize("K", [32, 160, 8224])
def test_large_activations(P, pairs, K):
    # scales 2^-9, 3 2^-9, 2^-6 and zero: terms up to 6 * 2^-6 |x|; K of them stay under 2^127
    top = min(3.3e38, 2.0 ** 127 * 2.0 ** 6 / (6 * K) * 0.98)
    check(P, pairs, K, [0x01, 0x03, 0x08, 0x00], values(pairs, K, 0.5 * top, top, 5))
    top = min(3.3e38, 2.0 ** 127 * 2.0 ** 9 / (6 * K) * 0.98)
    check(P, pairs, K, [0x01], values(pairs, K, 0.9 * top, top, 6))
    check(P, pairs, K, [0x00], values(pairs, K, 3.0e38, 3.38e38, 7))      # zeros times the largest values: zeros
    # scales up to 448 and activations that leave the sums just inside
    top = 2.0 ** 127 / (6 * 448 * K) * 0.98
    check(P, pairs, K, [0x7E, 0x38, 0x01], values(pairs, K, 0.5 * top, top, 8))


@pytest.mark.parametrize("pairs", [1, 2, 3, 17])
@pytest.mark.parametrize("K", [32, 160, 8224])
@pytest.mark.parametrize("low,high", [(0.0, 2.0 ** -126), (2.0 ** -126, 2.0 ** -124), (2.0 ** -118, 2.0 ** -116)])
def test_small_activations(P, pairs, K, low, high):
    x = values(pairs, K, low, high, 9)
    for scales in ([0x01], [0x7E], [0x01, 0x08, 0x38, 0x55, 0x7E, 0x00]):
        check(P, pairs, K, scales, x)


@pytest.mark.parametrize("pairs", [1, 2, 3])
def test_every_scale(P, pairs):
    """Each of the 127 scale bytes that are values, alone."""
    K, N = 128, 64
    x = values(pairs, K, 0.5, 2.0, 11)
    for byte in range(127):
        wq, w = weights(P, N, K, [byte], byte)
        y, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
        got = P.moe_gemv_nvfp4(x, wq, N, epilogue=P.EPI_F32)
        assert ((got.double() - y).abs() <= (K + 3) * U * mag + U * 1.02 * y.abs()).all(), hex(byte)
    wq, _ = weights(P, N, K, [0x7F], 3)
    assert torch.isnan(P.moe_gemv_nvfp4(x, wq, N, epilogue=P.EPI_F32)).all()
