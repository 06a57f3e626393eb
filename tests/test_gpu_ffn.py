"""swiglu_ffn_fwd / _bwd against fp64.

Tolerances, with u = 2^-24 and b = 2^-8 (half a bf16 step). A product of K terms accumulates in fp32:
off by at most (K + 2) u sum|terms|, whatever the order. The activation's exponential and reciprocal
are off by at most 16 u (1 + |h1|) of the value. Values rounded to bf16 between the products carry
b of themselves, propagated through the next product with absolute values:
    E_h  = (H + 2) u |x| |w13|^T                     (before h is stored)
    E_a  = b |a| + 16 u (1 + |h1|) |a| + 1.1 (E_h1 |h3| + E_h3 |h1|) (|silu'| < 1.1, |silu(h)| <= |h|)
    E_y  = E_a |w2|^T + (F + 2) u |a| |w2|^T (+ u |y|), and b |y| for the store
and in the same way backwards. The bound on E_a uses first-order terms; 1.02 covers the rest.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U, B = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def mk(shape, std, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def case(M, H, F, seed, add=True):
    return dict(x=mk((M, H), 1.0, seed), w13=mk((2 * F, H), 1.2 / H ** 0.5, seed + 1), w2=mk((H, F), F ** -0.5, seed + 2),
                add=mk((M, H), 0.5, seed + 3) if add else None)


def D(c, k):
    return c[k].double()


def ref_fwd(c):
    """On the device of c's tensors, in fp64."""
    F = c["w2"].shape[1]
    x, w13, w2 = D(c, "x"), D(c, "w13"), D(c, "w2")
    H = x.shape[1]
    h = x @ w13.t()
    eh = (H + 2) * U * (x.abs() @ w13.abs().t())
    h1, h3 = h[:, :F], h[:, F:]
    sg = torch.sigmoid(h1)
    a = h1 * sg * h3
    ea = B * a.abs() + 16 * U * (1 + h1.abs()) * a.abs() + 1.1 * (eh[:, :F] * h3.abs() + eh[:, F:] * h1.abs())
    y = a @ w2.t()
    ey = ea @ w2.abs().t() + (F + 2) * U * (a.abs() @ w2.abs().t())
    if c["add"] is not None:
        y = y + D(c, "add")
    return h, 1.02 * eh + (B + U) * h.abs(), y, 1.02 * ey + (B + 2 * U) * y.abs()


def within(got, ref, bound, what):
    bad = ~((got.to(ref.device).double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside the bound, first at {bad.nonzero()[0].tolist()}"


def dev(c):
    return {k: None if v is None else v.to(DEV) for k, v in c.items()}


# one token to several tiles, sizes around every tile edge, contraction lengths that end inside a
# stage, features and columns that are multiples of 8 only
SHAPES = [(1, 64, 32), (1, 512, 136), (2, 1000, 264), (3, 8, 8), (7, 256, 64), (15, 320, 40), (16, 512, 512),
          (17, 776, 128), (33, 1024, 72), (45, 520, 256), (63, 264, 328), (64, 1024, 256), (65, 136, 128), (100, 512, 520),
          (127, 256, 128), (129, 264, 136), (200, 96, 600), (255, 520, 264), (257, 640, 384), (300, 1032, 40),
          (513, 256, 256), (700, 512, 648)]


@pytest.mark.parametrize("M,H,F", SHAPES)
def test_forward(P, M, H, F):
    c = case(M, H, F, M + H + F, add=(M + F // 8) % 2 == 0)
    d = dev(c)
    h, hb, y, yb = ref_fwd(c)
    got, h13 = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], add=d["add"], save_h13=True)
    within(h13, h, hb, "h13")
    within(got, y, yb, "y")
    bare, none = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], add=d["add"])
    assert none is None and torch.equal(bare, got)
    if c["add"] is not None:
        buf = d["add"].clone()
        P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], add=buf, out=buf)
        assert torch.equal(buf, got)


def bwd_case(M, H, F, seed):
    c = case(M, H, F, seed, add=False)
    c["dy"] = mk((M, H), 1.0, seed + 7)
    c["h13"] = mk((M, 2 * F), 1.2, seed + 8)
    return c


def ref_bwd(c):
    F = c["w2"].shape[1]
    x, w13, w2, dy, h = (D(c, k) for k in ("x", "w13", "w2", "dy", "h13"))
    M, H = x.shape
    h1, h3 = h[:, :F], h[:, F:]
    s = torch.sigmoid(h1)
    d1 = s * (1 + h1 * (1 - s))
    a = h1 * s * h3
    ea = (B + 16 * U * (1 + h1.abs())) * a.abs()
    da = dy @ w2
    eda = (H + 2) * U * (dy.abs() @ w2.abs())
    dh = torch.cat([da * h3 * d1, da * h1 * s], 1)
    # the elementary functions: 16 u (1 + |h1|) of s and of 1 - s, hence of each factor's terms
    f1 = 16 * U * (1 + h1.abs()) * (s * (1 + h1.abs() * (1 - s)) + s * h1.abs())
    edh = torch.cat([eda * (h3 * d1).abs() + (da * h3).abs() * f1, eda * (h1 * s).abs() + 16 * U * (1 + h1.abs()) * (da * h1 * s).abs()], 1)
    edh = 1.02 * edh + (B + U) * dh.abs()
    out = {"dx": (dh @ w13, edh @ w13.abs() + (2 * F + 2) * U * (dh.abs() @ w13.abs())),
           "dw13": (dh.t() @ x, edh.t() @ x.abs() + (M + 2) * U * (dh.abs().t() @ x.abs())),
           "dw2": (dy.t() @ a, dy.abs().t() @ ea + (M + 2) * U * (dy.abs().t() @ a.abs()))}
    return {k: (r, 1.02 * e) for k, (r, e) in out.items()}


@pytest.mark.parametrize("M,H,F", SHAPES)
def test_backward(P, M, H, F):
    c = bwd_case(M, H, F, M + H + F)
    d = dev(c)
    ref = ref_bwd(c)
    args = (d["dy"], d["x"], d["w13"], d["w2"], d["h13"])
    for dt, half in ((torch.float32, 0.0), (torch.bfloat16, B)):
        got = dict(zip(("dx", "dw13", "dw2"), P.swiglu_ffn_bwd(*args, dw_dtype=dt)))
        for k, (r, e) in ref.items():
            extra = (B if k == "dx" else half) + U
            within(got[k], r, e + extra * (r.abs() + e), f"{k} {dt}")
    only = P.swiglu_ffn_bwd(*args, flags=P.BWD_DGRAD)
    assert torch.equal(only[0], got["dx"]) and only[1] is None and only[2] is None
    only = P.swiglu_ffn_bwd(*args, flags=P.BWD_WGRAD, dw_dtype=torch.bfloat16)
    assert only[0] is None and torch.equal(only[1], got["dw13"]) and torch.equal(only[2], got["dw2"])


def test_backward_against_differences(P):
    """Central differences of sum(dy y) in fp64 along random directions of x, w1 || w3 and w2. h13 is
    the forward's, so its rounding to bf16 (b of each h) joins the bound: it moves the gradients by the
    second derivatives, at most 1.1 |da| (|h3| + 1) b (|h1| + |h3|) in each of dh1, dh3."""
    M, H, F, h = 9, 96, 40, 1e-4
    c = case(M, H, F, 5, add=False)
    d = dev(c)
    dy = mk((M, H), 1.0, 77)
    _, h13 = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], save_h13=True)
    got = P.swiglu_ffn_bwd(dy.to(DEV), d["x"], d["w13"], d["w2"], h13)
    c.update(dy=dy, h13=h13.cpu())
    ref = ref_bwd(c)
    hh = h13.double().cpu()
    h1, h3 = hh[:, :F].abs(), hh[:, F:].abs()
    da = (dy.double() @ D(c, "w2")).abs()
    e = torch.cat([1.1 * da * (h3 + 1) * B * (h1 + h3)] * 2, 1) * 1.1
    ea = 1.2 * B * (h1 * h3) * 2
    more = {"dx": e @ D(c, "w13").abs(), "dw13": e.t() @ D(c, "x").abs(), "dw2": dy.double().abs().t() @ ea}

    def loss(x, w13, w2):
        z = x @ w13.t()
        return float((dy.double() * ((z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:]) @ w2.t())).sum())

    base = [D(c, "x"), D(c, "w13"), D(c, "w2")]
    for i, (k, name) in enumerate((("dx", "x"), ("dw13", "w13"), ("dw2", "w2"))):
        v = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64) * base[i].std()
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - h * v, base[i] + h * v
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        g = got[i].double().cpu()
        bound = ((ref[k][1] + more[k] + (B if k == "dx" else 0) * g.abs() + 2 * U * g.abs()) * v.abs()).sum()
        # cut-off h^2 / 6 of a third derivative below 1e4, rounding 1e-16 / h of the terms
        assert abs(num - float((g * v).sum())) <= float(bound) + 1e4 * h * h / 6 + 1e-9


def test_rows_are_independent_and_repeatable(P):
    """A row's result does not depend on what stands in other rows (infinities and NaN there stay there),
    and a call repeats bit for bit."""
    c = case(70, 512, 256, 9)
    d = dev(c)
    y0, h0 = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], add=d["add"], save_h13=True)
    y1, h1 = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], add=d["add"], save_h13=True)
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    x = d["x"].clone()
    x[3] = float("nan")
    x[69, 5] = float("inf")
    y2, h2 = P.swiglu_ffn_fwd(x, d["w13"], d["w2"], add=d["add"], save_h13=True)
    keep = [i for i in range(70) if i not in (3, 69)]
    assert torch.equal(y2[keep], y0[keep]) and torch.equal(h2[keep], h0[keep])
    assert torch.isnan(y2[3]).all() and not torch.isfinite(h2[69]).any()


def test_no_tokens(P):
    c = dev(bwd_case(0, 64, 32, 1))
    y, h13 = P.swiglu_ffn_fwd(c["x"], c["w13"], c["w2"], save_h13=True)
    assert y.shape == (0, 64) and h13.shape == (0, 64)
    for dt in (torch.float32, torch.bfloat16):
        dw = [torch.full(s, 7.0, dtype=dt, device=DEV) for s in ((64, 64), (64, 32))]
        dx, a, b = P.swiglu_ffn_bwd(c["dy"], c["x"], c["w13"], c["w2"], c["h13"], dw_dtype=dt, dw13=dw[0], dw2=dw[1])
        assert dx.shape == (0, 64) and (a == 0).all() and (b == 0).all()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_neighbouring_memory_is_left_alone(P, M):
    """Outputs inside larger buffers: what lies before and behind them keeps its bytes."""
    H, F = 264, 72
    c = bwd_case(M, H, F, 12)
    d = dev(c)

    def guarded(shape, dt):
        n = shape[0] * shape[1]
        buf = torch.full((n + 512,), 3.0, dtype=dt, device=DEV)
        return buf, buf[256:256 + n].view(shape)

    bufs = [guarded((M, H), torch.bfloat16), guarded((2 * F, H), torch.float32), guarded((H, F), torch.float32)]
    ws = [torch.full((P.swiglu_ffn_fwd_workspace_size(M, H, F) + 512,), 9, dtype=torch.uint8, device=DEV),
          torch.full((P.swiglu_ffn_bwd_workspace_size(M, H, F) + 512,), 9, dtype=torch.uint8, device=DEV)]
    y, _ = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], out=bufs[0][1], workspace=ws[0][:-512])
    assert torch.equal(y, P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"])[0])
    P.swiglu_ffn_bwd(d["dy"], d["x"], d["w13"], d["w2"], d["h13"], dw13=bufs[1][1], dw2=bufs[2][1], workspace=ws[1][:-512])
    for buf, _ in bufs:
        assert (buf[:256] == 3).all() and (buf[-256:] == 3).all()
    for w in ws:
        assert (w[-512:] == 9).all()


@pytest.mark.parametrize("M", [1, 50, 300])
def test_streams_and_graph(P, M):
    """On another stream, and captured once and replayed with other inputs between eager work."""
    c = dev(bwd_case(M, 512, 256, 31))

    def call():
        y, h13 = P.swiglu_ffn_fwd(c["x"], c["w13"], c["w2"], save_h13=True)
        return (y, h13, *P.swiglu_ffn_bwd(c["dy"], c["x"], c["w13"], c["w2"], h13))

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
        c["x"].copy_(torch.randn((M, 512), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call())), f"replay {k}"


# sizes around the 256 x 256 tiles (128 of them and more; 1300 rows have 66 and take 128 x 128 ones), ragged
# at every edge; 4200 and 4260 rows have 289, the last 33 in halves of 128 rows, with 104 rows of the last
# one left or 164; fp64 on the GPU
@pytest.mark.parametrize("M,H,F", [(2600, 264, 2056), (2600, 4104, 72), (1300, 2056, 1288), (4260, 4104, 72),
                                   (4200, 4104, 72), (4200, 72, 2056)])
def test_forward_of_many_tiles(P, M, H, F):
    d = dev(case(M, H, F, M + H + F))
    h, hb, y, yb = ref_fwd(d)
    got, h13 = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], add=d["add"], save_h13=True)
    within(h13, h, hb, "h13")
    within(got, y, yb, "y")


@pytest.mark.parametrize("M,H,F", [(5000, 2600, 2056), (5000, 5000, 1032), (3000, 264, 136), (9000, 72, 264), (4200, 72, 4104)])
def test_backward_of_many_tiles(P, M, H, F):
    d = dev(bwd_case(M, H, F, M + H + F))
    ref = ref_bwd(d)
    for dt, half in ((torch.float32, 0.0), (torch.bfloat16, B)):
        got = dict(zip(("dx", "dw13", "dw2"), P.swiglu_ffn_bwd(d["dy"], d["x"], d["w13"], d["w2"], d["h13"], dw_dtype=dt)))
        for k, (r, e) in ref.items():
            within(got[k], r, e + ((B if k == "dx" else half) + U) * (r.abs() + e), f"{k} {dt}")


def test_offsets_past_32_bits(P):
    """300000 rows of 7168 (2.15 G values, 4.3 GB): the last rows against fp64, the rows just past 2^31
    values too, and the weights' gradients of a dy that is zero but in those rows."""
    M, H, F = 300_000, 7168, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((M, H), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    c = case(8, H, F, 3, add=False)
    d = dict(w13=c["w13"].to(DEV), w2=c["w2"].to(DEV))
    y, h13 = P.swiglu_ffn_fwd(x, d["w13"], d["w2"], save_h13=True)
    rows = torch.cat([torch.arange(299_590, 299_600), torch.arange(M - 40, M)]).to(DEV)
    part = dict(d, x=x[rows].clone(), add=None)
    h, hb, yr, yb = ref_fwd(part)
    within(h13[rows], h, hb, "h13")
    within(y[rows], yr, yb, "y")
    dy = y.zero_()
    dy[rows] = torch.empty((50, H), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    dx, dw13, dw2 = P.swiglu_ffn_bwd(dy, x, d["w13"], d["w2"], h13)
    ref = ref_bwd(dict(part, dy=dy[rows].clone(), h13=h13[rows].clone()))
    within(dx[rows], ref["dx"][0], ref["dx"][1] + (B + U) * (ref["dx"][0].abs() + ref["dx"][1]), "dx")
    assert (dx[:1000] == 0).all()
    # M terms in the sums, all but 50 of them zero: exact
    for k, got in (("dw13", dw13), ("dw2", dw2)):
        within(got, ref[k][0], ref[k][1] + U * ref[k][0].abs(), k)
