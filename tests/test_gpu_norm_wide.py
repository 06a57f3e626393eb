"""The norm where a workgroup takes several wide rows, and its outputs to the last bits.

Tolerances, with u = 2^-24. rstd: squares are summed in fp64, so without a residual it is the exact value
rounded (u, and 2^-40 for the sum); z's own rounding with a residual adds u. y and its 8-bit codes carry
the errors of s and of the product z s, so what is rounded is off by the last rounding u, 2^-20 u for the
terms left out, and with a residual 2 u more for z's and for what z's rounding does to s: without one every
code is the nearest of the exact y, but where y lies within 1.01 u of itself of a tie.
Backward: as the products stand in the formula, |dz - ref| <= 64 u (s (|t| + |xh| S) + |dres|) + half a
step, S = mean |t xh|, for the dot product's serial 32 squares, 6 butterfly steps and 16 wavefronts.
dgamma: a thread adds the terms of the rows that its workgroup takes, then 3 groups of a workgroup, then 1
of 32 threads the partial rows that fall to it, then 32 sums: with G workgroups of r rows at a time
(rows / (G r) + 1 + 3 + G / 32 + 32 + 3) u sum |dy xh|, the last 3 for each term's own products.
"""
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


def within(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside the bound, first at {bad.nonzero()[0].tolist()}"


def stream_like(rows, cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.randn((rows, cols), generator=g, device=DEV)
    t[:, :: max(cols // 8, 1)] *= 12.0
    return t * torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV)), g


def groups(rows, cols):
    """Rows that a workgroup takes at a time, and the number of workgroups."""
    r = 4 if cols <= 2048 else 1
    return r, min(-(-rows // r), 256 if cols > 4096 and rows <= 1024 else 512)


# every width of a thread group and number of pieces, with more rows than one round of workgroups takes
@pytest.mark.parametrize("rows,cols", [(9001, 96), (4101, 1000), (2600, 1032), (5001, 2048), (1100, 4096), (2050, 2056),
                                       (777, 7168), (1024, 4104), (1025, 8200), (520, 16384), (600, 16392), (1537, 5000)])
@pytest.mark.parametrize("zt,dt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_backward_of_more_rows_than_workgroups(P, rows, cols, zt, dt):
    z, g = stream_like(rows, cols, cols)
    z = z.to(zt)
    gamma = 1.0 + 0.1 * torch.randn(cols, generator=g, device=DEV)
    rstd = (1.0 / torch.sqrt((z.double() ** 2).mean(1) + 1e-6)).float()
    # a mean far from zero: the terms of dgamma share a sign with xh's, and their sum grows with the rows
    dy = (1e-3 * (torch.randn((rows, cols), generator=g, device=DEV) + torch.sign(z.float()))).to(dt)
    dres = (1e-3 * torch.randn((rows, cols), generator=g, device=DEV)).to(zt) if rows % 2 else None
    dz, dgamma = P.rmsnorm_residual_bwd(dy, z, gamma, rstd, dres=dres)
    s = rstd.double()[:, None]
    xh, t = z.double() * s, dy.double() * gamma.double()
    ref = s * (t - xh * (t * xh).mean(1, keepdim=True))
    bound = s * (t.abs() + xh.abs() * (t * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        ref, bound = ref + dres.double(), bound + dres.double().abs()
    within(dz, ref, 64 * U * bound + (HALF[zt] + U) * ref.abs(), "dz")
    r, G = groups(rows, cols)
    term = dy.double() * xh
    within(dgamma, term.sum(0), (rows / (G * r) + 1 + 3 + G / 32 + 32 + 3) * U * term.abs().sum(0), "dgamma")
    again = P.rmsnorm_residual_bwd(dy, z, gamma, rstd, dres=dres)
    assert torch.equal(again[0], dz) and torch.equal(again[1], dgamma)


def test_dgamma_of_many_wide_rows(P):
    """300000 rows of 7168 (offsets past 32 bits): dgamma against an fp64 sum taken in pieces."""
    M, C = 300_000, 7168
    g = torch.Generator(device=DEV).manual_seed(5)
    z = torch.empty((M, C), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    dy = torch.empty((M, C), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    gamma = torch.ones(C, device=DEV)
    rstd = torch.rand(M, generator=g, device=DEV) + 0.5
    dgamma = P.rmsnorm_residual_bwd(dy, z, gamma, rstd, dz=torch.empty_like(z))[1]
    ref, size = torch.zeros(C, dtype=torch.float64, device=DEV), torch.zeros(C, dtype=torch.float64, device=DEV)
    for i in range(0, M, 10_000):
        term = dy[i:i + 10_000].double() * z[i:i + 10_000].double() * rstd[i:i + 10_000].double()[:, None]
        ref += term.sum(0)
        size += term.abs().sum(0)
    within(dgamma, ref, (M / 512 + 1 + 3 + 16 + 32 + 3) * U * size, "dgamma")


def nearest_codes(y):
    """Scale exponents and E4M3 values (to nearest) of y fp64 [blocks, 32], with the step at each value."""
    amax = y.abs().amax(1, keepdim=True)
    e = torch.ceil(torch.log2(amax / 448.0))
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
    t = y / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
    return e.squeeze(1), t, step


@pytest.mark.parametrize("rows,cols", [(8000, 2048), (4000, 4096), (2300, 7168)])
@pytest.mark.parametrize("res", [None, torch.float32])
def test_outputs_to_the_last_bits(P, rows, cols, res):
    """16 million codes, some 50 of them within 4 u of a tie: only those within the bound may be the
    neighbour. rstd to its rounding."""
    slack = 1.01 * U if res is None else 3.01 * U
    s, g = stream_like(rows, cols, 9)
    gamma = 1.0 + 0.1 * torch.randn(cols, generator=g, device=DEV)
    x = (s if res is None else 0.3 * torch.randn((rows, cols), generator=g, device=DEV)).to(torch.bfloat16)
    o = P.rmsnorm_residual_fwd(x, gamma, 1e-6, residual=None if res is None else s, want_mxfp8=True, want_rstd=True)
    z = x.double() if res is None else x.double() + s.double()
    rs = 1.0 / torch.sqrt((z * z).mean(1) + 1e-6)
    within(o.rstd, rs, slack * rs, "rstd")
    y = z.mul_(rs[:, None]).mul_(gamma.double()).view(-1, 32)
    e, t, step = nearest_codes(y)
    got = o.codes.view(torch.float8_e4m3fn).double().view(-1, 32)
    # a block's scale may be the neighbour's only where its largest value lies within the bound of 448 2^e
    other = (o.e8m0.view(-1).double() - 127) != e
    top = (y.abs().amax(1) / (448.0 * torch.exp2(e)))[other]
    assert (torch.minimum((top - 1).abs(), (2 * top - 1).abs()) <= 2 * slack).all()
    same = ~other
    within(got[same], t[same], step[same] / 2 + slack * t[same].abs(), "codes")


def test_infinite_gamma_and_norms_past_the_range(P):
    """An infinite gamma makes its column infinite or NaN and leaves the others alone; a row whose
    1 / norm passes fp32 (eps 0, zeros or subnormals) has an infinite rstd and is NaN, the other rows are
    what they are."""
    rows, cols = 9, 264
    s, g = stream_like(rows, cols, 3)
    x = s.to(torch.bfloat16)
    gamma = 1.0 + 0.1 * torch.randn(cols, generator=g, device=DEV)
    odd = gamma.clone()
    odd[8], odd[263] = float("inf"), -float("inf")
    a, b = P.rmsnorm_residual_fwd(x, gamma), P.rmsnorm_residual_fwd(x, odd)
    keep = torch.isfinite(odd)
    assert torch.equal(a.y[:, keep], b.y[:, keep]) and not torch.isfinite(b.y[:, ~keep]).any()
    x[3], x[7] = 0.0, 1e-40
    a = P.rmsnorm_residual_fwd(x, gamma, 0.0, want_rstd=True)
    rest = [0, 1, 2, 4, 5, 6, 8]
    alone = P.rmsnorm_residual_fwd(x[rest].contiguous(), gamma, 0.0)
    assert torch.equal(a.y[rest], alone.y) and torch.isfinite(alone.y).all()
    assert torch.isinf(a.rstd[[3, 7]]).all() and torch.isnan(a.y[[3, 7]]).all()
