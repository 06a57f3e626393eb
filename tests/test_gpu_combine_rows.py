"""moe_combine_rows_fwd / _bwd against fp64.

Tolerances, with u = 2^-24: a sum of k + 1 terms of fma is off by at most (k + 2) u sum|terms|, a dot product of H
terms by (H + 2) u sum|terms|; a stored value adds half a step of its type (2^-8 for bf16, u for fp32)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def mk(shape, std, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def within(got, ref, bound, what):
    bound = bound + (U if got.dtype == torch.float32 else 2.0 ** -8) * 1.02 * ref.abs()
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside the bound, first at {bad.nonzero()[0].tolist()}"


def slots(T, k, M, seed, outside=False):
    """Distinct slots of [0, M), some pairs (outside) with none."""
    g = torch.Generator().manual_seed(seed)
    s = torch.randperm(M, generator=g)[:T * k].view(T, k).to(torch.int32)
    if outside:
        drop = torch.rand((T, k), generator=g) < 0.3
        s[drop] = torch.tensor([-1, M, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64)[torch.randint(0, 4, (int(drop.sum()),), generator=g)].to(torch.int32)
    return s.to(DEV)


def ref_fwd(y, so, gates, add):
    M, H = y.shape
    T, k = so.shape
    on = (so >= 0) & (so < M)
    rows = y.double()[so.long().clamp(0, max(M - 1, 0))] if M else torch.zeros((T, k, H), dtype=torch.float64, device=DEV)
    g = (torch.ones((T, k), dtype=torch.float64, device=DEV) if gates is None else gates.double()) * on
    t = torch.where(on[:, :, None], rows, 0.0) * g[:, :, None]
    out, mag = t.sum(1), t.abs().sum(1)
    if add is not None:
        out, mag = out + add.double(), mag + add.double().abs()
    return out, (k + 2) * U * mag


SHAPES = [(1, 1, 8, 1), (3, 2, 64, 6), (7, 8, 520, 60), (16, 9, 1024, 160), (5, 64, 136, 320), (129, 4, 2056, 600),
          (2, 3, 8192, 9), (300, 8, 4096, 2400), (1, 17, 16392, 20)]


@pytest.mark.parametrize("T,k,H,M", SHAPES)
@pytest.mark.parametrize("ydt", DTYPES)
def test_forward(P, T, k, H, M, ydt):
    y = mk((M, H), 1.0, T + H, ydt)
    add = mk((T, H), 0.5, T + H + 1, torch.bfloat16)
    gates = mk((T, k), 1.0, T + H + 2, torch.float32)
    for outside in (False, True):
        so = slots(T, k, M, T + k, outside)
        for odt in DTYPES:
            for gt in (gates, None):
                for ad in (add, None):
                    ref, e = ref_fwd(y, so, gt, ad)
                    got = P.moe_combine_rows_fwd(y, so, gt, ad, out_dtype=odt)
                    within(got, ref, e, f"outside {outside} out {odt}")
    so = slots(T, k, M, T + k)
    buf = add.clone()
    P.moe_combine_rows_fwd(y, so, gates, buf, out=buf)
    assert torch.equal(buf, P.moe_combine_rows_fwd(y, so, gates, add))
    # the same slot for every pair: read as often as it is named
    same = torch.full((T, k), M - 1, dtype=torch.int32, device=DEV)
    ref, e = ref_fwd(y, same, gates, None)
    within(P.moe_combine_rows_fwd(y, same, gates), ref, e, "one slot")


@pytest.mark.parametrize("T,k,H,M", SHAPES)
@pytest.mark.parametrize("ydt", DTYPES)
@pytest.mark.parametrize("ddt", DTYPES)
def test_backward(P, T, k, H, M, ydt, ddt):
    y = mk((M, H), 1.0, T + H, ydt)
    dout = mk((T, H), 1.0, T + H + 3, ddt)
    gates = mk((T, k), 1.0, T + H + 2, torch.float32)
    for outside in (False, True):
        so = slots(T, k, M, T + k, outside)
        on = (so >= 0) & (so < M)
        for gt in (gates, None):
            g = (torch.ones_like(gates) if gt is None else gates).double()
            dy = torch.full((M, H), 3.0, dtype=ydt, device=DEV)
            _, dg = P.moe_combine_rows_bwd(dout, y, so, gt, dy=dy)
            want = torch.full((M, H), 3.0, dtype=torch.float64, device=DEV)
            want[so[on].long()] = (g[:, :, None] * dout.double()[:, None, :])[on]
            within(dy, want, U * want.abs(), "dy")
            named = torch.zeros(M, dtype=torch.bool, device=DEV)
            named[so[on].long()] = True
            assert (dy[~named] == 3.0).all()
            t = y.double()[so.long().clamp(0, M - 1)] * dout.double()[:, None, :] * on[:, :, None]
            within(dg, t.sum(2), (H + 2) * U * t.abs().sum(2), "dgates")
            assert (dg[~on] == 0).all()
            only, none = P.moe_combine_rows_bwd(dout, y, so, gt, want_dgates=False, dy=torch.full_like(dy, 3.0))
            assert none is None and torch.equal(only, dy)
            none, only = P.moe_combine_rows_bwd(dout, y, so, gt, want_dy=False)
            assert none is None and torch.equal(only, dg)


def test_rows_without_a_pair_are_zeros_by_default(P):
    y, dout = mk((9, 64), 1.0, 1, torch.float32), mk((2, 64), 1.0, 2, torch.float32)
    so = slots(2, 3, 9, 3)
    dy, _ = P.moe_combine_rows_bwd(dout, y, so)
    rest = torch.ones(9, dtype=torch.bool, device=DEV)
    rest[so.flatten().long()] = False
    assert (dy[rest] == 0).all() and not (dy[~rest] == 0).all()


def test_nothing_to_do(P):
    y = mk((4, 64), 1.0, 1, torch.bfloat16)
    none = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    assert P.moe_combine_rows_fwd(y, none).shape == (0, 64)
    dy, dg = P.moe_combine_rows_bwd(torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV), y, none)
    assert (dy == 0).all() and dg.shape == (0, 3)
    empty = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    so = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    add = mk((2, 64), 1.0, 2, torch.bfloat16)
    assert (P.moe_combine_rows_fwd(empty, so) == 0).all() and torch.equal(P.moe_combine_rows_fwd(empty, so, add=add), add)
    dy, dg = P.moe_combine_rows_bwd(add, empty, so)
    assert dy.shape == (0, 64) and (dg == 0).all()


def test_backward_of_no_rows(P):
    empty = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    dy, dg = P.moe_combine_rows_bwd(empty, empty, torch.zeros((0, 3), dtype=torch.int32, device=DEV))
    assert dy.shape == (0, 64) and dg.shape == (0, 3)
    out = torch.ones((2, 64), dtype=torch.bfloat16, device=DEV)
    dy, dg = P.moe_combine_rows_bwd(out, empty, torch.zeros((2, 3), dtype=torch.int32, device=DEV), want_dgates=False)
    assert dy.shape == (0, 64) and dg is None


def test_checked_indices(P, monkeypatch):
    """With CHECK_INDICES a slot named twice, and a new dy with rows that no pair writes, are refused."""
    monkeypatch.setattr(P, "CHECK_INDICES", True)
    y, dout = mk((6, 64), 1.0, 1, torch.float32), mk((2, 64), 1.0, 2, torch.float32)
    so = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32, device=DEV)
    P.moe_combine_rows_bwd(dout, y, so)
    so[1, 2] = -1
    with pytest.raises(P.PmnError):
        P.moe_combine_rows_bwd(dout, y, so)
    dy = torch.zeros_like(y)
    P.moe_combine_rows_bwd(dout, y, so, dy=dy)
    assert (dy[5] == 0).all()
    so[1, 2] = 0
    with pytest.raises(P.PmnError):
        P.moe_combine_rows_bwd(dout, y, so, dy=dy)


def test_a_slots_nan_stays_with_its_token(P):
    y, so = mk((40, 136), 1.0, 1, torch.bfloat16), slots(10, 4, 40, 2)
    gates = mk((10, 4), 1.0, 3, torch.float32)
    bad = y.clone()
    bad[so[6, 2].long()] = float("nan")
    a, b = P.moe_combine_rows_fwd(y, so, gates), P.moe_combine_rows_fwd(bad, so, gates)
    keep = torch.arange(10, device=DEV) != 6
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[6]).all()
    # a dropped pair's row is not read: NaN behind it, and a NaN gate, do nothing
    so2, g2 = so.clone(), gates.clone()
    so2[6, 2], g2[6, 2] = -1, float("nan")
    assert torch.isfinite(P.moe_combine_rows_fwd(bad, so2, g2)).all()


def test_streams_and_replayed_graph(P):
    y, so = mk((120, 264), 1.0, 1, torch.bfloat16), slots(30, 4, 120, 2)
    gates, dout = mk((30, 4), 1.0, 3, torch.float32), mk((30, 264), 1.0, 4, torch.bfloat16)
    run = lambda: [P.moe_combine_rows_fwd(y, so, gates), *P.moe_combine_rows_bwd(dout, y, so, gates)]  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for r in range(4):
        so.copy_(slots(30, 4, 120, 50 + r))
        y.copy_(mk((120, 264), 1.0, 60 + r, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), r


def test_offsets_past_32_bits(P):
    """Rows past 2^32 bytes: 600000 rows of 4096 bf16 (4.9 GB)."""
    y = torch.zeros((600000, 4096), dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([[599999, 0], [540000, 300000]], dtype=torch.int32, device=DEV)
    y[at.flatten().long()] = mk((4, 4096), 1.0, 1, torch.bfloat16)
    gates = mk((2, 2), 1.0, 2, torch.float32)
    small = y[at.flatten().long()]
    local = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    assert torch.equal(P.moe_combine_rows_fwd(y, at, gates), P.moe_combine_rows_fwd(small, local, gates))
    dout = mk((2, 4096), 1.0, 3, torch.bfloat16)
    dy, dg = P.moe_combine_rows_bwd(dout, y, at, gates)
    dy2, dg2 = P.moe_combine_rows_bwd(dout, small, local, gates)
    assert torch.equal(dy[at.flatten().long()], dy2) and torch.equal(dg, dg2)
    assert int((dy != 0).any(1).sum()) == 4
