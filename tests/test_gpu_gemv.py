"""moe_gemv_nvfp4 against fp64 on the dequantized weights.

Tolerances, with u = 2^-24 and b = 2^-8. fp4 * e4m3 is exact in bf16 and its products with bf16 activations are exact
in fp32; the sum of K of them is off by at most (K + 2) u sum|terms|, the outer scale adds u. A bf16 output adds b,
an fp32 one u. With gates: u for gate * outer and one more for its product, and one for each of k and the added row.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U, B = 2.0 ** -24, 2.0 ** -8
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def mk(shape, std, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(DEV)


def weights(P, G, N, K, seed, per=None):
    return P.nvfp4_quantize(mk((G * N, K), 0.02, seed), P.NVFP4_WEIGHT, rows_per_outer=per or N)


def values(wq):
    """fp64 values of an NVFP4 matrix."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=DEV)
    c = wq.codes.long()
    v = torch.stack([grid[c % 16], grid[c // 16]], 2).flatten(1)
    s = wq.scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    return v * s * wq.outer.double().repeat_interleave(wq.rows_per_outer)[:, None]


def ref_pairs(x, w, ids, N, G):
    """(y, bound) [T, k, N] of x [T, K] or [T, k, K]; ids outside [0, G): zeros."""
    T, k = ids.shape
    K = x.shape[-1]
    x = x.double() if x.dim() == 3 else x.double()[:, None, :].expand(T, k, K)
    y = torch.zeros((T, k, N), dtype=torch.float64, device=DEV)
    e = torch.zeros_like(y)
    for g in range(G):
        t, j = (ids == g).nonzero(as_tuple=True)
        wg = w[g * N:(g + 1) * N]
        y[t, j] = x[t, j] @ wg.t()
        e[t, j] = (K + 3) * U * (x[t, j].abs() @ wg.abs().t())
    return y, e


def within(got, ref, bound, what):
    bound = bound + (U if got.dtype == torch.float32 else B) * 1.02 * ref.abs()
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside the bound, first at {bad.nonzero()[0].tolist()}"


def choose(T, k, G, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, G), generator=g).topk(k, 1).indices.to(torch.int32).to(DEV)


def check(P, T, k, G, N, K, ids, per_pair, seed, per=None):
    wq = weights(P, G, N, K, seed, per)
    w = values(wq)
    x = mk((T, k, K) if per_pair else (T, K), 1.0, seed + 1)
    y, e = ref_pairs(x, w, ids, N, G)
    for epi in (P.EPI_F32, P.EPI_BF16):
        within(P.moe_gemv_nvfp4(x, wq, N, ids, epi), y, e, f"y {epi}")
    if N % 64 == 0:
        h1, h3 = y.chunk(2, 2)
        e1, e3 = e.chunk(2, 2)
        a = h1 * torch.sigmoid(h1) * h3
        ea = 1.02 * (16 * U * (1 + h1.abs()) * a.abs() + 1.1 * (e1 * h3.abs() + e3 * h1.abs()))
        within(P.moe_gemv_nvfp4(x, wq, N, ids, P.EPI_SWIGLU), a, ea, "swiglu")
    gates = torch.rand((T, k), generator=torch.Generator().manual_seed(seed + 2)).to(DEV)
    add = mk((T, N), 0.5, seed + 3)
    gd = gates.double()[:, :, None]
    s = (y * gd).sum(1)
    es = (e * gd).sum(1) + (k + 4) * U * ((y.abs() * gd).sum(1) + add.double().abs())
    for epi in (P.EPI_F32, P.EPI_BF16):
        within(P.moe_gemv_nvfp4(x, wq, N, ids, epi, gates=gates), s, es, f"sum {epi}")
        within(P.moe_gemv_nvfp4(x, wq, N, ids, epi, gates=gates, add=add), s + add.double(), es, f"sum + add {epi}")


# tokens around the tiles of 16 and 64 columns, pairs below and above the experts, contractions that end in
# a unit of 128 with 32, 64 or 96 left and shorter than one, rows of one workgroup to several
@pytest.mark.parametrize("T,k,G,N,K", [
    (1, 1, 1, 32, 32), (1, 1, 1, 64, 7168), (1, 8, 48, 128, 1056), (1, 3, 3, 192, 96), (2, 4, 9, 64, 544),
    (5, 8, 16, 448, 2048), (15, 2, 40, 64, 160), (16, 16, 16, 64, 288), (17, 3, 4, 96, 1120), (33, 8, 12, 64, 384),
    (64, 8, 48, 128, 640), (61, 1, 1, 256, 512), (70, 2, 2, 64, 224), (130, 1, 1, 64, 128), (256, 16, 20, 64, 64),
    (3, 20, 24, 64, 96), (40, 5, 300, 32, 64), (1, 2, 3, 64, 8224), (4, 1, 2, 64, 16480), (9, 2, 2, 32, 17280)])
@pytest.mark.parametrize("per_pair", [False, True])
def test_pairs_and_sums(P, T, k, G, N, K, per_pair):
    check(P, T, k, G, N, K, choose(T, k, G, T + k), per_pair, 7 * T + G + K)


def test_dense(P):
    for T in (1, 7, 16, 45, 100):
        wq = weights(P, 1, 320, 416, T)
        x = mk((T, 416), 1.0, T + 1)
        y, e = ref_pairs(x, values(wq), torch.zeros((T, 1), dtype=torch.int32, device=DEV), 320, 1)
        got = P.moe_gemv_nvfp4(x, wq, 320, epilogue=P.EPI_F32)
        assert got.shape == (T, 320)
        within(got, y[:, 0], e[:, 0], f"dense {T}")
        gates = torch.full((T, 1), 0.5, device=DEV)
        within(P.moe_gemv_nvfp4(x, wq, 320, gates=gates), 0.5 * y[:, 0], e[:, 0] + 6 * U * y[:, 0].abs(), "dense, gated")


@pytest.mark.parametrize("per", [32, 64, 192])
def test_outer_scales_of_fewer_rows(P, per):
    check(P, 4, 2, 3, 192, 160, choose(4, 2, 3, 1), False, 77, per=per)


@pytest.mark.parametrize("T", [1, 6, 16, 30])
def test_repeated_and_outside_ids(P, T):
    """The same expert several times in a token, and ids that name none: zeros, and nothing in the sums."""
    G, k = 5, 6
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-2, G + 2, (T, k), generator=g).to(torch.int32)
    ids[0] = torch.tensor([2, 2, -1, 2, 7, 2], dtype=torch.int32)
    check(P, T, k, G, 64, 352, ids.to(DEV), True, 100 + T)
    check(P, T, k, G, 64, 352, ids.to(DEV), False, 200 + T)
    none = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    check(P, T, k, G, 64, 352, none, True, 300 + T)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_an_outside_pairs_gate_is_not_read(P, value):
    G, k, N, K = 5, 4, 64, 352
    wq, x = weights(P, G, N, K, 31), mk((6, K), 1.0, 32)
    ids = choose(6, k, G, 33)
    ids[0, 1], ids[3], ids[5, 3] = -1, G, 1 << 30
    gates = torch.rand((6, k), generator=torch.Generator().manual_seed(34)).to(DEV)
    bad = torch.where((ids < 0) | (ids >= G), torch.full_like(gates, value), gates)
    a, b = (P.moe_gemv_nvfp4(x, wq, N, ids, P.EPI_F32, gates=g) for g in (gates, bad))
    assert torch.isfinite(b).all() and torch.equal(a, b) and (b[3] == 0).all()


def test_tokens_keep_to_themselves(P):
    """A token's NaN or infinity reaches its own rows only, and an expert's NaN scale the tokens that name it."""
    T, k, G, N, K = 9, 3, 6, 64, 256
    wq = weights(P, G, N, K, 5)
    x, ids = mk((T, K), 1.0, 6), choose(T, k, G, 7)
    gates = torch.rand((T, k), generator=torch.Generator().manual_seed(8)).to(DEV)
    calls = [lambda a, q: P.moe_gemv_nvfp4(a, q, N, ids), lambda a, q: P.moe_gemv_nvfp4(a, q, N, ids, gates=gates)]
    keep = torch.arange(T, device=DEV) != 4
    for value in (float("nan"), float("inf")):
        bad = x.clone()
        bad[4, 100] = value
        for f in calls:
            a, b = f(x, wq), f(bad, wq)
            assert torch.equal(a[keep], b[keep]) and not torch.isfinite(b[4]).all()
    q = P.NVFP4(wq.codes, wq.scales.clone(), wq.outer, wq.rows_per_outer)
    q.scales[2 * N:3 * N] = 0x7F
    uses = (ids == 2).any(1)
    assert uses.any() and not uses.all()
    for f in calls:
        a, b = f(x, wq), f(x, q)
        assert torch.equal(a[~uses], b[~uses]) and torch.isnan(b[uses]).flatten(1).any(1).all()


@pytest.mark.parametrize("T", [2, 16, 40])
def test_one_column_does_not_depend_on_the_others(P, T):
    """A token's rows are the same bits whatever the other tokens' activations are, and as another token of the batch
    (pairs of an expert are summed alike; how many there are chooses the instructions)."""
    G, N, K, k = 8, 128, 1056, 2
    wq = weights(P, G, N, K, 9)
    x, ids = mk((T, K), 1.0, 10), choose(T, k, G, 11)
    whole = P.moe_gemv_nvfp4(x, wq, N, ids, P.EPI_F32)
    for t in (0, T // 2, T - 1):
        other = mk((T, K), 1.0, 12)
        other[t] = x[t]
        assert torch.equal(P.moe_gemv_nvfp4(other, wq, N, ids, P.EPI_F32)[t], whole[t])
    back = torch.arange(T - 1, -1, -1, device=DEV)
    assert torch.equal(P.moe_gemv_nvfp4(x[back].contiguous(), wq, N, ids[back].contiguous(), P.EPI_F32)[back], whole)


def test_memory_around_the_outputs(P):
    T, k, G, N, K = 5, 3, 7, 96, 160
    wq, x, ids = weights(P, G, N, K, 13), mk((T, K), 1.0, 14), choose(T, k, G, 15)
    gates = torch.rand((T, k), device=DEV)
    for shape, kw in (((T, k, N), {}), ((T, N), dict(gates=gates))):
        n = torch.Size(shape).numel()
        buf = torch.full((n + 512,), 3.0, dtype=torch.bfloat16, device=DEV)
        P.moe_gemv_nvfp4(x, wq, N, ids, out=buf[256:256 + n].view(shape), **kw)
        assert (buf[:256] == 3.0).all() and (buf[256 + n:] == 3.0).all() and not (buf[256:256 + n] == 3.0).all()


def test_streams_and_replayed_graph(P):
    T, k, G, N, K = 20, 4, 6, 128, 416
    wq, x, ids = weights(P, G, N, K, 17), mk((T, K), 1.0, 18), choose(T, k, G, 19)
    gates = torch.rand((T, k), device=DEV)
    run = lambda: [P.moe_gemv_nvfp4(x, wq, N, ids, P.EPI_SWIGLU), P.moe_gemv_nvfp4(x, wq, N, ids, gates=gates),  # noqa: E731
                   P.moe_gemv_nvfp4(x[:3], wq, N, ids[:3], gates=gates[:3])]
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
        ids.copy_(choose(T, k, G, 30 + r))
        x.copy_(mk((T, K), 1.0, 40 + r))
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), r


def test_as_many_pairs_as_there_may_be(P):
    """4096 pairs of a contraction as long as LDS holds, in three tiles a workgroup."""
    T, k, G, N, K = 512, 8, 48, 2048, 8192
    wq, x, ids = weights(P, G, N, K, 25), mk((T, K), 1.0, 26), choose(T, k, G, 27)
    y, e = ref_pairs(x, values(wq), ids, N, G)
    within(P.moe_gemv_nvfp4(x, wq, N, ids, P.EPI_F32), y, e, "y")
    h1, h3 = y.chunk(2, 2)
    e1, e3 = e.chunk(2, 2)
    a = h1 * torch.sigmoid(h1) * h3
    within(P.moe_gemv_nvfp4(x, wq, N, ids, P.EPI_SWIGLU), a,
           1.02 * (16 * U * (1 + h1.abs()) * a.abs() + 1.1 * (e1 * h3.abs() + e3 * h1.abs())), "swiglu")


def test_two_calls_at_once(P):
    """Calls with gates on two streams share nothing (each brings its workspace)."""
    G, N, K, k = 8, 256, 1056, 3
    wq = weights(P, G, N, K, 29)
    cs = [(mk((T, K), 1.0, T), choose(T, k, G, T), torch.rand((T, k), generator=torch.Generator().manual_seed(T)).to(DEV))
          for T in (5, 24)]
    run = lambda c: P.moe_gemv_nvfp4(c[0], wq, N, c[1], gates=c[2])  # noqa: E731
    want = [run(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(run(c))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_weights_past_32_bits(P):
    """Codes past 2^32 bytes: 100 experts of 4096 x 22016 (4.5 GB)."""
    G, N, K = 100, 4096, 22016
    codes = torch.zeros((G * N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((G * N, K // 16), dtype=torch.uint8, device=DEV)
    one = P.nvfp4_quantize(mk((N, K), 0.02, 23), P.NVFP4_WEIGHT, rows_per_outer=N)
    for g in (1, 98):
        codes[g * N:(g + 1) * N], scales[g * N:(g + 1) * N] = one.codes, one.scales
    wq = P.NVFP4(codes, scales, one.outer.expand(G).contiguous(), N)
    x = mk((2, K), 1.0, 24)
    ids = torch.tensor([[98, 3], [1, 98]], dtype=torch.int32, device=DEV)
    y = P.moe_gemv_nvfp4(x, wq, N, ids, P.EPI_F32)
    want = P.moe_gemv_nvfp4(x, one, N, epilogue=P.EPI_F32)
    assert torch.equal(y[0, 0], want[0]) and torch.equal(y[1, 0], want[1]) and torch.equal(y[1, 1], want[1])
    assert (y[0, 1] == 0).all() and want.abs().max() > 0
