"""rmsnorm_residual_fwd / _bwd against fp64.

Tolerances, with u = 2^-24. Forward: wide enough for sums in fp32 (at most 32 squares a thread, 6
butterfly steps and 16 wavefronts, z itself off by u: 57 u of the sum, 32 u of 1 / sqrt; z's rounding and
two products in y: 40 u in all); the kernel's are in fp64, and test_gpu_norm_wide.py holds them to it.
Stored values add half a step of their type (bf16 2^-8, fp32 u; E4M3 2^-4, or 2^-10 of the block's scale
below its normal range). Backward: the row's dot product is off by at most 60 u of S = mean|t xh|, so
|dz - ref| <= 64 u (s (|t| + |xh| S) + |dres|) + half a step; dgamma adds the rows that a thread takes (of
those tested here at most 3 of 2048 values and less, one of more), 3 groups of a workgroup, up to 16
partial rows and 32 sums: 128 u sum|dy xh| covers them.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def stream_like(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn((rows, cols), generator=g, dtype=torch.float64)
    t[:, :: max(cols // 8, 1)] *= 12.0
    return t * torch.exp(0.5 * torch.randn((rows, 1), generator=g, dtype=torch.float64))


def inputs(rows, cols, res, seed):
    g = torch.Generator().manual_seed(seed + 1)
    gamma = (1.0 + 0.1 * torch.randn(cols, generator=g)).float()
    s = stream_like(rows, cols, seed)
    if res is None:
        return s.to(torch.bfloat16), None, gamma
    return torch.randn((rows, cols), generator=g).to(torch.bfloat16), s.to(res), gamma


def ref_fwd(x, r, gamma, eps):
    z = x.double() + (0 if r is None else r.double())
    s = 1.0 / torch.sqrt((z * z).mean(1) + eps)
    return z, s, z * s[:, None] * gamma.double()


def gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def within(got, ref, bound, what):
    bad = (got.to(ref.device).double() - ref).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside the bound, first at {bad.nonzero()[0].tolist()}"


def check_codes(codes, e8m0, y):
    rows, cols = y.shape
    v = codes.cpu().view(torch.float8_e4m3fn).double().view(rows, -1, 32)
    e = e8m0.cpu().double() - 127.0
    b = y.view(rows, -1, 32)
    amax = b.abs().amax(-1)
    assert (amax <= 448.0 * torch.exp2(e) * (1 + 40 * U)).all(), "a block is larger than its scale holds"
    smaller = (amax > 448.0 * torch.exp2(e - 1) * (1 - 40 * U)) | (e == -127)
    assert smaller.all(), "a block's scale is not the smallest"
    sc = torch.exp2(e)[..., None]
    within(v * sc, b, 2.0 ** -4 * b.abs().clamp_min(2.0 ** -6 * sc) * (1 + 40 * U) + 40 * U * b.abs(), "codes")


CASES = [(1, 8), (3, 40), (1, 7168), (5, 512), (9, 1000), (130, 1024), (7, 2048), (6, 2056), (37, 4096), (4, 5000),
         (3, 6152), (2, 8192), (5, 8200), (3, 16384), (2, 32768), (1031, 96)]


@pytest.mark.parametrize("rows,cols", CASES)
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
def test_forward(P, rows, cols, res):
    """Every split of a row (one wavefront, 256 and 1024 threads, each piece count, ragged ends) and
    each residual type."""
    x, r, gamma = inputs(rows, cols, res, 100 + cols)
    z, s, y = ref_fwd(x, r, gamma, 1e-6)
    mx = cols % 32 == 0
    xd, rd, gd = gpu(x, r, gamma)
    o = P.rmsnorm_residual_fwd(xd, gd, 1e-6, residual=rd, want_mxfp8=mx, want_rstd=True)
    within(o.y, y, (2.0 ** -8 + 40 * U) * y.abs(), "y")
    within(o.rstd, s, 40 * U * s, "rstd")
    if res is None:
        assert o.z is None
    else:
        assert o.z.dtype == res
        within(o.z, z, (HALF[res] + 2 * U) * z.abs(), "z")
    if mx:
        check_codes(o.codes, o.e8m0, y)
        only = P.rmsnorm_residual_fwd(xd, gd, 1e-6, residual=rd, want_y=False, want_mxfp8=True)
        assert only.y is None and torch.equal(only.codes, o.codes) and torch.equal(only.e8m0, o.e8m0)


def test_forward_rows_that_are_special(P):
    """A zero row, a row of one value, subnormal and large values, infinities and NaN: each row is by
    itself, a zero row gives zeros, and what is not finite is NaN in both outputs, never a number."""
    cols = 256
    x = torch.randn((8, cols), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    x[0] = 0
    x[1] = 0
    x[1, 5] = 3.0
    x[2] *= 2.0 ** -70
    x[3] *= 2.0 ** 50
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    gamma = torch.ones(cols)
    xd, gd = gpu(x, gamma)
    o = P.rmsnorm_residual_fwd(xd, gd, 1e-6, want_mxfp8=True, want_rstd=True)
    z, s, y = ref_fwd(x, None, gamma, 1e-6)
    ok = [0, 1, 2, 3, 6, 7]
    within(o.y[ok], y[ok], (2.0 ** -8 + 40 * U) * y[ok].abs() + 2.0 ** -133, "y")
    check_codes(o.codes[[0, 1, 3, 6, 7]], o.e8m0[[0, 1, 3, 6, 7]], y[[0, 1, 3, 6, 7]])
    assert (o.codes[0] == 0).all() and (o.e8m0[0] == 0).all()
    v = o.codes.view(torch.float8_e4m3fn).float()
    assert torch.isnan(o.y[4, 7]) and torch.isnan(v[4, 7]) and (o.y[4, :7] == 0).all()
    assert torch.isnan(o.y[5]).all() and torch.isnan(v[5]).all()
    alone = P.rmsnorm_residual_fwd(xd[6:8].contiguous(), gd, 1e-6, want_mxfp8=True)
    assert torch.equal(alone.codes, o.codes[6:8]) and torch.equal(alone.y, o.y[6:8])


def test_forward_in_place_and_no_rows(P):
    x, r, gamma = inputs(33, 512, torch.float32, 7)
    xd, rd, gd = gpu(x, r, gamma)
    a = P.rmsnorm_residual_fwd(xd, gd, residual=rd)
    keep = rd.clone()
    b = P.rmsnorm_residual_fwd(xd, gd, residual=keep, z_out=keep)
    assert b.z is keep and torch.equal(a.z, keep) and torch.equal(a.y, b.y)
    e = P.rmsnorm_residual_fwd(xd[:0], gd, residual=rd[:0], want_mxfp8=True, want_rstd=True)
    assert e.y.shape == (0, 512) and e.codes.shape == (0, 512)


def ref_bwd(dy, z, gamma, rstd, dres):
    dy, z, s = dy.double(), z.double(), rstd.double()[:, None]
    xh, t = z * s, dy * gamma.double()
    dz = s * (t - xh * (t * xh).mean(1, keepdim=True))
    bound = s * (t.abs() + xh.abs() * (t * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        dz, bound = dz + dres.double(), bound + dres.double().abs()
    return dz, 64 * U * bound, (dy * xh).sum(0), 128 * U * (dy * xh).abs().sum(0)


@pytest.mark.parametrize("rows,cols", CASES + [(2500, 64), (4099, 128)])
@pytest.mark.parametrize("zt,dt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_backward(P, rows, cols, zt, dt):
    z = stream_like(rows, cols, 30 + cols).to(zt)
    g = torch.Generator().manual_seed(cols)
    gamma = (1.0 + 0.1 * torch.randn(cols, generator=g)).float()
    rstd = (1.0 / torch.sqrt((z.double() ** 2).mean(1) + 1e-6)).float()
    dy = (1e-3 * torch.randn((rows, cols), generator=g)).to(dt)
    dres = (1e-3 * torch.randn((rows, cols), generator=g)).to(zt) if rows % 2 else None
    ref, bound, dg, dgb = ref_bwd(dy, z, gamma, rstd, dres)
    d = gpu(dy, z, gamma, rstd, dres)
    dz, dgamma = P.rmsnorm_residual_bwd(d[0], d[1], d[2], d[3], dres=d[4])
    assert dz.dtype == zt
    within(dz, ref, bound + (HALF[zt] + U) * ref.abs(), "dz")
    within(dgamma, dg, dgb + U * dg.abs(), "dgamma")
    again = P.rmsnorm_residual_bwd(d[0], d[1], d[2], d[3], dres=d[4])
    assert torch.equal(again[0], dz) and torch.equal(again[1], dgamma)
    if dres is not None:
        same = d[4].clone()
        P.rmsnorm_residual_bwd(d[0], d[1], d[2], d[3], dres=same, dz=same)
        assert torch.equal(same, dz)


def test_backward_against_differences(P):
    """Central differences of sum(dy y) in fp64 along random directions of z and gamma: off by the
    kernel's own bounds, and by the differences' cut-off, h^2 / 6 of a third derivative that stays
    below 1e3 here, and their rounding, 1e-16 / h of the sum."""
    rows, cols, h = 6, 320, 1e-4
    z = stream_like(rows, cols, 3).float()
    g = torch.Generator().manual_seed(8)
    gamma = (1.0 + 0.1 * torch.randn(cols, generator=g)).float()
    dy = torch.randn((rows, cols), generator=g).float()
    rstd = (1.0 / torch.sqrt((z.double() ** 2).mean(1) + 1e-6)).float()
    d = gpu(dy, z, gamma, rstd)
    dz, dgamma = P.rmsnorm_residual_bwd(*d)
    _, zb, _, gb = ref_bwd(dy, z, gamma, rstd, None)

    def loss(zz, gg):
        s = 1.0 / torch.sqrt((zz * zz).mean(1, keepdim=True) + 1e-6)
        return float((dy.double() * zz * s * gg).sum())

    for seed in range(3):
        q = torch.Generator().manual_seed(50 + seed)
        vz = torch.randn(z.shape, generator=q, dtype=torch.float64)
        vg = torch.randn(cols, generator=q, dtype=torch.float64)
        Z, G = z.double(), gamma.double()
        slack = 1e3 * h * h / 6 + 1e-16 / h * float((dy.double().abs() * 4).sum())
        num = (loss(Z + h * vz, G) - loss(Z - h * vz, G)) / (2 * h)
        ana = float((dz.double().cpu() * vz).sum())
        assert abs(num - ana) <= float(((zb + 2 * U * dz.cpu().double().abs()) * vz.abs()).sum()) + slack
        num = (loss(Z, G + h * vg) - loss(Z, G - h * vg)) / (2 * h)
        ana = float((dgamma.double().cpu() * vg).sum())
        assert abs(num - ana) <= float(((gb + 8 * U * dgamma.cpu().double().abs()) * vg.abs()).sum()) + slack


def test_backward_of_no_rows_is_zero(P):
    z = torch.empty((0, 64), device=DEV)
    dz, dg = P.rmsnorm_residual_bwd(z, z, torch.ones(64, device=DEV), torch.empty(0, device=DEV))
    assert dz.shape == (0, 64) and (dg == 0).all()


def test_streams_and_graph(P):
    """On another stream, and captured once and replayed with other inputs between eager work."""
    x, r, gamma = inputs(300, 1024, torch.bfloat16, 21)
    xd, rd, gd = gpu(x, r, gamma)
    dy = torch.randn((300, 1024), device=DEV).to(torch.bfloat16)

    def call():
        o = P.rmsnorm_residual_fwd(xd, gd, residual=rd, want_mxfp8=True, want_rstd=True)
        return (*P.rmsnorm_residual_bwd(dy, o.z, gd, o.rstd), o.y, o.codes, o.e8m0)

    eager = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for k in range(3):
        xd.copy_(torch.randn((300, 1024), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call())), f"replay {k}"


def test_offsets_past_32_bits(P):
    """300000 rows of 7168 (2.15 G values): the rows just past 2^31 values and the last ones."""
    M, C = 300_000, 7168
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.empty((M, C), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    r = torch.empty((M, C), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    gamma = torch.ones(C, device=DEV)
    o = P.rmsnorm_residual_fwd(x, gamma, residual=r, want_mxfp8=True, want_rstd=True)
    rows = torch.cat([torch.arange(299_590, 299_600), torch.arange(M - 10, M)]).to(DEV)
    few = P.rmsnorm_residual_fwd(x[rows].contiguous(), gamma, residual=r[rows].contiguous(), want_mxfp8=True, want_rstd=True)
    for k in ("y", "z", "codes", "e8m0", "rstd"):
        assert torch.equal(getattr(o, k)[rows], getattr(few, k)), k
    del x, r
    z = o.z[rows].contiguous()
    dz, _ = P.rmsnorm_residual_bwd(o.y, o.z, gamma, o.rstd)
    again, _ = P.rmsnorm_residual_bwd(few.y, z, gamma, few.rstd)
    assert torch.equal(dz[rows], again)


def test_more_rows_than_a_launch_holds(P):
    """2^26 + 5 rows of 8 values are more than 2^32 threads in all: rows at the ends, around the border
    of two launches (2^25) and a random choice against the same rows alone."""
    M, C = (1 << 26) + 5, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty((M, C), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    gamma = torch.linspace(0.5, 1.5, C, device=DEV)
    o = P.rmsnorm_residual_fwd(x, gamma, want_rstd=True)
    rows = torch.cat([torch.arange(8), torch.arange((1 << 25) - 8, (1 << 25) + 8), torch.arange(M - 16, M),
                      torch.randint(0, M, (100_000,), generator=torch.Generator().manual_seed(4))]).to(DEV)
    few = P.rmsnorm_residual_fwd(x[rows].contiguous(), gamma, want_rstd=True)
    assert torch.equal(o.y[rows], few.y) and torch.equal(o.rstd[rows], few.rstd)
