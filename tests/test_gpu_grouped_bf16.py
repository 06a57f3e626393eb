"""moe_grouped_gemm_fwd_bf16 / _bwd_bf16 against fp64.

Tolerances, with u = 2^-24 and b = 2^-8 (half a bf16 step). Products of bf16 values are exact in fp32; a sum of K
of them in fp32 is off by at most (K + 2) u sum|terms|, whatever its order. A bf16 output adds b, an fp32 one u of
the value. The activation's exponential and reciprocal are off by at most 16 u (1 + |h1|) of each factor they enter;
a first-order bound, with 1.02 for the rest.
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
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(DEV)


def offsets_of(counts):
    return torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int64, device=DEV)


def case(counts, N, K, seed, tokens=0):
    M, G = sum(counts), len(counts)
    g = torch.Generator().manual_seed(seed + 9)
    gather = torch.randint(0, tokens, (M,), generator=g).to(torch.int32).to(DEV) if tokens else None
    return dict(counts=counts, M=M, N=N, K=K, G=G, off=offsets_of(counts), gather=gather,
                x=mk((tokens or M, K), 1.0, seed), w=mk((G * N, K), 1.2 / K ** 0.5, seed + 1),
                dy=mk((M, N), 1.0, seed + 2))


def rows_of(c):
    return (c["x"] if c["gather"] is None else c["x"][c["gather"].long()]).double()


def groups(c):
    a = 0
    for g, n in enumerate(c["counts"]):
        yield g, a, a + n, c["w"][g * c["N"]:(g + 1) * c["N"]].double()
        a += n


def ref_y(c):
    x = rows_of(c)
    y = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device=DEV)
    e = torch.zeros_like(y)
    for g, a, b, w in groups(c):
        y[a:b] = x[a:b] @ w.t()
        e[a:b] = (c["K"] + 2) * U * (x[a:b].abs() @ w.abs().t())
    return y, e


def ref_bwd(c):
    x, dy = rows_of(c), c["dy"].double()
    da = torch.zeros((c["M"], c["K"]), dtype=torch.float64, device=DEV)
    dw = torch.zeros((c["G"] * c["N"], c["K"]), dtype=torch.float64, device=DEV)
    eda, edw = torch.zeros_like(da), torch.zeros_like(dw)
    for g, a, b, w in groups(c):
        da[a:b] = dy[a:b] @ w
        eda[a:b] = (c["N"] + 2) * U * (dy[a:b].abs() @ w.abs())
        r = slice(g * c["N"], (g + 1) * c["N"])
        dw[r] = dy[a:b].t() @ x[a:b]
        edw[r] = (b - a + 2) * U * (dy[a:b].abs().t() @ x[a:b].abs())
    return da, eda, dw, edw


def within(got, ref, bound, what):
    bound = bound + (U if got.dtype == torch.float32 else B) * 1.02 * ref.abs()
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside the bound, first at {bad.nonzero()[0].tolist()}"


def ref_swiglu(y, e):
    h1, h3 = y.chunk(2, 1)
    e1, e3 = e.chunk(2, 1)
    a = h1 * torch.sigmoid(h1) * h3
    return a, 1.02 * (16 * U * (1 + h1.abs()) * a.abs() + 1.1 * (e1 * h3.abs() + e3 * h1.abs()))


# group sizes around every unit's edge (16, 64, 128, 256 and their halves), empty groups first, last and in runs,
# over 64 groups; widths and contractions that are multiples of 8 only; a mean that takes each tile
CASES = [([1], 32, 64, 0), ([0, 3, 0, 16, 17, 0], 48, 72, 0), ([5, 0, 0, 1], 264, 1000, 9), ([2] * 70, 80, 136, 33),
         ([33, 0, 64, 65, 1], 144, 264, 0), ([40, 20, 90, 0], 520, 328, 77), ([100, 128, 129, 64], 272, 136, 0),
         ([130, 0, 127, 1, 200], 136, 520, 300), ([256, 257, 128, 385, 0, 300], 528, 264, 0),
         ([700, 3, 511], 256, 96, 0), ([300, 129, 384, 640], 784, 1032, 500), ([1025], 264, 2056, 0),
         ([0] * 66 + [20], 64, 64, 0), ([9, 14, 3, 30], 1040, 4104, 21),
         # enough tiles of a long contraction for the 256 x 256 ones, whole and half, and for 128 x 128 ones
         ([4000, 0, 129, 2500, 1, 1250, 1120], 1040, 4104, 0), ([3000, 128, 0, 1500, 257, 4115], 1040, 4104, 2000),
         ([(i * 37) % 125 for i in range(48)], 1040, 4104, 700), ([300 + (i * 61) % 97 for i in range(40)], 784, 1032, 0),
         ([2600, 5, 1400], 2064, 520, 900)]
IDS = [f"{len(c[0])}x{sum(c[0])}-{c[1]}x{c[2]}-{c[3]}" for c in CASES]


@pytest.mark.parametrize("counts,N,K,tokens", CASES, ids=IDS)
def test_forward(P, counts, N, K, tokens):
    c = case(counts, N, K, N + K, tokens)
    y, e = ref_y(c)
    for epi in (P.EPI_F32, P.EPI_BF16):
        within(P.moe_grouped_gemm_fwd_bf16(c["x"], c["w"], c["off"], c["M"], N, epi, gather=c["gather"]), y, e, f"y {epi}")
    if N % 16 != 0:
        return                                   # F = N / 2 features, a multiple of 8
    a, ea = ref_swiglu(y, e)
    got, h13 = P.moe_grouped_gemm_fwd_bf16(c["x"], c["w"], c["off"], c["M"], N, P.EPI_SWIGLU, gather=c["gather"],
                                           save_h13=True)
    within(h13, y, e, "h13")
    within(got, a, ea, "a")
    bare, none = P.moe_grouped_gemm_fwd_bf16(c["x"], c["w"], c["off"], c["M"], N, P.EPI_SWIGLU, gather=c["gather"])
    assert none is None and torch.equal(bare, got)


@pytest.mark.parametrize("counts,N,K,tokens", CASES, ids=IDS)
def test_backward(P, counts, N, K, tokens):
    c = case(counts, N, K, N + K + 1, tokens)
    da, eda, dw, edw = ref_bwd(c)
    args = (c["dy"], c["x"], c["w"], c["off"], c["M"], N)
    g32, w32 = P.moe_grouped_gemm_bwd_bf16(*args, gather=c["gather"], da_dtype=torch.float32)
    within(g32, da, eda, "da fp32")
    within(w32, dw, edw, "dw fp32")
    g16, none = P.moe_grouped_gemm_bwd_bf16(*args, flags=P.BWD_DGRAD, gather=c["gather"])
    assert none is None
    within(g16, da, eda, "da bf16")
    none, w16 = P.moe_grouped_gemm_bwd_bf16(*args, flags=P.BWD_WGRAD, gather=c["gather"], db_dtype=torch.bfloat16)
    assert none is None
    within(w16, dw, edw, "dw bf16")


# (a sum in parts rounds a value no more often than in one)
@pytest.mark.parametrize("counts,N,K,tokens", [([4767], 304, 960, 681), ([9000, 0, 5, 6000], 136, 264, 0), ([1, 33, 6000], 72, 136, 50),
                                               ([2500], 8, 8, 0), ([20000, 13000], 48, 40, 3000), ([2100] * 20, 128, 128, 0)])
def test_weight_gradients_in_parts(P, counts, N, K, tokens):
    """Few and small matrices over many slots: the contraction is split, also in replays that share a workspace."""
    c = case(counts, N, K, N + K + 7, tokens)
    M, G = c["M"], c["G"]
    need = P.moe_grouped_gemm_bwd_bf16_workspace_size(M, G, N, K, P.BWD_WGRAD, False)
    assert need >= 2 * G * N * K * 4
    _, _, dw, edw = ref_bwd(c)
    args = (c["dy"], c["x"], c["w"], c["off"], M, N)
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
    for dt in (torch.float32, torch.bfloat16):
        _, got = P.moe_grouped_gemm_bwd_bf16(*args, flags=P.BWD_WGRAD, gather=c["gather"], db_dtype=dt, workspace=ws[:need])
        within(got, dw, edw, f"dw {dt}")
        _, own = P.moe_grouped_gemm_bwd_bf16(*args, gather=c["gather"], db_dtype=dt)
        assert torch.equal(got, own)
    assert (ws[need:] == 0xFF).all()
    with pytest.raises(P.PmnError):
        P.moe_grouped_gemm_bwd_bf16(*args, gather=c["gather"], workspace=ws[:need - 1])
    run = lambda: P.moe_grouped_gemm_bwd_bf16(*args, flags=P.BWD_WGRAD, gather=c["gather"], workspace=ws[:need])[1]  # noqa: E731
    graphs, held = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(run())
        graphs.append(graph)
    for r in range(3):
        c["dy"].copy_(mk((M, N), 1.0, 60 + r))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(want, h) for h in held), r


@pytest.mark.parametrize("counts,N,K", [([6000, 0, 1700], 64, 136), ([3000], 40, 64)])
def test_weight_gradients_in_parts_of_h13(P, counts, N, K):
    c = case(counts, N, K, 71)
    M = c["M"]
    h13 = mk((M, 2 * K), 1.2, 72)
    assert P.moe_grouped_gemm_bwd_bf16_workspace_size(M, c["G"], N, K, 3, True) > M * K * 2 + 512
    dh, dw = P.moe_grouped_gemm_bwd_bf16(c["dy"], None, c["w"], c["off"], M, N, h13=h13)
    h1, h3 = h13.double().chunk(2, 1)
    act = h1 * torch.sigmoid(h1) * h3
    ea = (B + 16 * U * (1 + h1.abs())) * 1.02 * act.abs()
    for g, a, b, _ in groups(c):
        dy = c["dy"][a:b].double()
        within(dw[g * N:(g + 1) * N], dy.t() @ act[a:b], dy.abs().t() @ ea[a:b] + 1.02 * (b - a + 2) * U * (dy.abs().t() @ act[a:b].abs()),
               f"dw, group {g}")
    only, _ = P.moe_grouped_gemm_bwd_bf16(c["dy"], None, c["w"], c["off"], M, N, flags=P.BWD_DGRAD, h13=h13)
    assert torch.equal(only, dh)


@pytest.mark.parametrize("counts,N,K", [(c[0], c[1], c[2]) for c in CASES], ids=IDS)
def test_backward_through_swiglu(P, counts, N, K):
    """With h13 the gradient is dh13; without x the activation is taken from h13."""
    c = case(counts, N, K, N + K + 2)
    M = c["M"]
    h13 = mk((M, 2 * K), 1.2, N + K + 5)
    h1, h3 = h13.double().chunk(2, 1)
    s = torch.sigmoid(h1)
    act = h1 * s * h3
    c["x"] = act.float().to(torch.bfloat16)
    da, eda, dw, edw = ref_bwd(c)
    d1 = s * (1 + h1 * (1 - s))
    dh = torch.cat([da * h3 * d1, da * h1 * s], 1)
    f1 = 16 * U * (1 + h1.abs()) * (s * (1 + h1.abs() * (1 - s)) + s * h1.abs())
    edh = 1.02 * torch.cat([eda * (h3 * d1).abs() + (da * h3).abs() * f1,
                            eda * (h1 * s).abs() + 16 * U * (1 + h1.abs()) * (da * h1 * s).abs()], 1)
    got, w = P.moe_grouped_gemm_bwd_bf16(c["dy"], c["x"], c["w"], c["off"], M, N, h13=h13)
    within(got, dh, edh, "dh13")
    within(w, dw, edw, "dw")
    # x rebuilt: the kernel's own rounding of silu(h1) h3, b of the value and 16 u (1 + |h1|) before it
    got2, w2 = P.moe_grouped_gemm_bwd_bf16(c["dy"], None, c["w"], c["off"], M, N, h13=h13)
    assert torch.equal(got, got2)
    ea = (B + 16 * U * (1 + h1.abs())) * 1.02 * act.abs()
    a0 = 0
    for g, n in enumerate(counts):
        r, sl = slice(g * N, (g + 1) * N), slice(a0, a0 + n)
        dy = c["dy"][sl].double()
        ref = dy.t() @ act[sl]
        within(w2[r], ref, dy.abs().t() @ ea[sl] + 1.02 * (n + 2) * U * (dy.abs().t() @ act[sl].abs()), f"dw of h13, group {g}")
        a0 += n
    only, none = P.moe_grouped_gemm_bwd_bf16(c["dy"], None, c["w"], c["off"], M, N, flags=P.BWD_DGRAD, h13=h13)
    assert none is None and torch.equal(only, got)


def test_no_slots(P):
    c = case([0, 0, 0], 64, 64, 3)
    y = P.moe_grouped_gemm_fwd_bf16(c["x"], c["w"], c["off"], 0, 64)
    assert y.shape == (0, 64)
    for dt in (torch.float32, torch.bfloat16):
        db = torch.full((3 * 64, 64), 7.0, dtype=dt, device=DEV)
        da, _ = P.moe_grouped_gemm_bwd_bf16(c["dy"], c["x"], c["w"], c["off"], 0, 64, db_dtype=dt, db=db)
        assert da.shape == (0, 64) and (db == 0).all()


@pytest.mark.parametrize("counts", [[7, 0, 9, 4], [20, 60, 33, 0], [90, 140, 70], [300, 200, 0, 410]])
def test_rows_keep_to_themselves(P, counts):
    """A row of NaN or infinities reaches its own outputs, and in the weight gradient its own group's, no others:
    tiles and contractions end inside the operands' neighbours."""
    c = case(counts, 144, 136, 11)
    M = c["M"]
    for value in (float("nan"), float("inf")):
        x, dy = c["x"].clone(), c["dy"].clone()
        first, last = 0, counts[0] - 1        # the last row of the first group
        x[last], dy[last] = value, value
        y0 = P.moe_grouped_gemm_fwd_bf16(c["x"], c["w"], c["off"], M, 144)
        y1 = P.moe_grouped_gemm_fwd_bf16(x, c["w"], c["off"], M, 144)
        keep = torch.arange(M, device=DEV) != last
        assert torch.equal(y0[keep], y1[keep]) and not torch.isfinite(y1[last]).any()
        da0, dw0 = P.moe_grouped_gemm_bwd_bf16(c["dy"], c["x"], c["w"], c["off"], M, 144)
        da1, dw1 = P.moe_grouped_gemm_bwd_bf16(dy, x, c["w"], c["off"], M, 144)
        assert torch.equal(da0[keep], da1[keep]) and not torch.isfinite(da1[last]).any()
        assert torch.equal(dw0[144:], dw1[144:]) and not torch.isfinite(dw1[:144]).any()


def test_memory_around_the_outputs(P):
    """Nothing outside the outputs is written, whatever the tiles' edges."""
    c = case([130, 3, 0, 50], 144, 72, 13)
    M, N, K = c["M"], 144, 72

    def guarded(n, dtype):
        buf = torch.full((n + 512,), 3.0, dtype=dtype, device=DEV)
        return buf, buf[256:256 + n]

    def intact(buf, n):
        assert (buf[:256] == 3.0).all() and (buf[256 + n:] == 3.0).all()

    for epi, dt in ((P.EPI_F32, torch.float32), (P.EPI_BF16, torch.bfloat16)):
        buf, out = guarded(M * N, dt)
        P.moe_grouped_gemm_fwd_bf16(c["x"], c["w"], c["off"], M, N, epi, out=out.view(M, N))
        intact(buf, M * N)
    buf, out = guarded(M * N // 2, torch.bfloat16)
    hbuf, h = guarded(M * N, torch.bfloat16)
    P.moe_grouped_gemm_fwd_bf16(c["x"], c["w"], c["off"], M, N, P.EPI_SWIGLU, out=out.view(M, N // 2), out_aux=h.view(M, N))
    intact(buf, M * N // 2)
    intact(hbuf, M * N)
    abuf, da = guarded(M * K, torch.bfloat16)
    wbuf, dw = guarded(4 * N * K, torch.float32)
    P.moe_grouped_gemm_bwd_bf16(c["dy"], c["x"], c["w"], c["off"], M, N, da=da.view(M, K), db=dw.view(4 * N, K))
    intact(abuf, M * K)
    intact(wbuf, 4 * N * K)


def test_streams_and_replayed_graph(P):
    c = case([40, 0, 300, 77], 272, 264, 17, tokens=200)
    M, N = c["M"], 272
    fwd = lambda: P.moe_grouped_gemm_fwd_bf16(c["x"], c["w"], c["off"], M, N, gather=c["gather"])  # noqa: E731
    bwd = lambda: P.moe_grouped_gemm_bwd_bf16(c["dy"], c["x"], c["w"], c["off"], M, N, gather=c["gather"])  # noqa: E731
    want = [fwd(), *bwd()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [fwd(), *bwd()]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [fwd(), *bwd()]
    # other sizes of the groups and other rows before each replay: both are read when the graph runs
    for r, counts in enumerate(([40, 0, 300, 77], [1, 400, 0, 16], [417, 0, 0, 0], [40, 0, 300, 77])):
        c["off"].copy_(offsets_of(counts))
        c["x"].copy_(mk(tuple(c["x"].shape), 1.0, 50 + r))
        graph.replay()
        torch.cuda.synchronize()
        want = [fwd(), *bwd()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), counts


def test_two_calls_at_once(P):
    """Calls on two streams share nothing."""
    cs = [case([200, 31, 150], 264, 520, s, tokens=90) for s in (21, 22)]
    run = lambda c: P.moe_grouped_gemm_bwd_bf16(c["dy"], c["x"], c["w"], c["off"], c["M"], 264, gather=c["gather"])  # noqa: E731
    want = [run(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(run(c))
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_offsets_past_32_bits(P):
    """Gathered rows and outputs past 2^32 bytes, weights past 2^31."""
    K, rows = 7168, 310000                     # 4.4 GB of rows
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 5, 150000, 299600, 309999], device=DEV)
    x[at] = mk((5, K), 1.0, 31)
    gather = at[[4, 0, 3, 2, 1, 4]].to(torch.int32)
    w = mk((2 * 64, K), 0.02, 32)
    off = offsets_of([4, 2])
    y = P.moe_grouped_gemm_fwd_bf16(x, w, off, 6, 64, P.EPI_F32, gather=gather)
    few = P.moe_grouped_gemm_fwd_bf16(x[gather.long()], w, off, 6, 64, P.EPI_F32)
    assert torch.equal(y, few) and y.abs().min() > 0
    dy = mk((6, 64), 1.0, 33)
    _, dw = P.moe_grouped_gemm_bwd_bf16(dy, x, w, off, 6, 64, gather=gather)
    _, dw2 = P.moe_grouped_gemm_bwd_bf16(dy, x[gather.long()], w, off, 6, 64)
    assert torch.equal(dw, dw2)
    # the same rows through the large tiles
    big = gather.repeat(60)
    y = P.moe_grouped_gemm_fwd_bf16(x, w[:64], offsets_of([360]), 360, 64, P.EPI_F32, gather=big)
    want = x[at].double() @ w[:64].double().t()
    place = torch.tensor([4, 0, 3, 2, 1, 4], device=DEV).repeat(60)
    bound = (K + 2) * U * (x[at].double().abs() @ w[:64].double().abs().t())
    within(y, want[place], bound[place], "gathered")
    del x
    M, N, K = 150000, 16384, 8                 # 4.9 GB of outputs
    x, w = mk((M, K), 1.0, 34), mk((2 * N, K), 1.0, 35)
    y = P.moe_grouped_gemm_fwd_bf16(x, w, offsets_of([149000, 1000]), M, N)
    for s, g in ((0, 0), (148999, 0), (149000, 1), (149999, 1)):
        want = x[s].double() @ w[g * N:(g + 1) * N].double().t()
        within(y[s], want, (K + 2) * U * (x[s].double().abs() @ w[g * N:(g + 1) * N].double().abs().t()), f"row {s}")


def test_gathered_weight_gradient_through_large_tiles_past_32_bits(P):
    """x rows past 2^32 bytes as gathered k of 256 x 256 tiles, groups without and with one slot between."""
    N, K, rows = 1040, 4104, 600000             # 4.9 GB of rows
    counts = [700, 0, 1, 3000, 1500, 900, 2000, 255]
    M = sum(counts)
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(51)
    at = torch.cat([torch.randint(0, rows, (997,), generator=g), torch.tensor([0, rows - 1, rows - 2])]).to(DEV)
    x[at] = mk((1000, K), 1.0, 52)
    gather = at[torch.randint(0, 1000, (M,), generator=g).to(DEV)].to(torch.int32)
    dy, w, off = mk((M, N), 1.0, 53), mk((8 * N, K), 0.02, 54), offsets_of(counts)
    _, dw = P.moe_grouped_gemm_bwd_bf16(dy, x, w, off, M, N, flags=P.BWD_WGRAD, gather=gather)
    _, dw2 = P.moe_grouped_gemm_bwd_bf16(dy, x[gather.long()], w, off, M, N, flags=P.BWD_WGRAD)
    assert torch.equal(dw, dw2) and dw.view(8, -1).abs().amax(1).gt(0).tolist() == [c > 0 for c in counts]


def test_gradients_agree_with_differences(P):
    """<dw, v> and <da, v> against central differences of the fp64 loss sum(y dy): the loss is bilinear, so a central
    difference is exact up to rounding; bounds as above, summed with |v|."""
    c = case([9, 0, 40, 21], 48, 64, 41)
    da, dw = P.moe_grouped_gemm_bwd_bf16(c["dy"], c["x"], c["w"], c["off"], c["M"], 48, da_dtype=torch.float32)
    _, eda, _, edw = ref_bwd(c)
    dy = c["dy"].double()

    def loss(x, w):
        return sum((x[a:b] @ w[g * 48:(g + 1) * 48].t() * dy[a:b]).sum() for g, a, b, _ in groups(c))

    x, w = c["x"].double(), c["w"].double()
    vx, vw = mk(tuple(x.shape), 1.0, 42).double(), mk(tuple(w.shape), 1.0, 43).double()
    t = 2.0 ** -10
    num_x = (loss(x + t * vx, w) - loss(x - t * vx, w)) / (2 * t)
    num_w = (loss(x, w + t * vw) - loss(x, w - t * vw)) / (2 * t)
    assert abs((da.double() * vx).sum() - num_x) <= ((eda + U * da.double().abs()) * vx.abs()).sum() + 1e-9 * num_x.abs()
    assert abs((dw.double() * vw).sum() - num_w) <= ((edw + U * dw.double().abs()) * vw.abs()).sum() + 1e-9 * num_w.abs()
