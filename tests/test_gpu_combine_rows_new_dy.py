"""moe_combine_rows_bwd without a given dy, and moe_rows_zero_unnamed: rows that no pair names are zeros, whatever
the new memory held. Copies and zeros are exact: no tolerances."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def slots(T, k, M, seed, drop):
    """Distinct slots of [0, M), a share of the pairs without one."""
    g = torch.Generator().manual_seed(seed)
    s = torch.randperm(M, generator=g)[:T * k].view(T, k)
    s[torch.rand((T, k), generator=g) < drop] = torch.tensor([-1, M, 2 ** 31 - 1, -2 ** 31])[seed % 4]
    return s.to(torch.int32).to(DEV)


def named(so, M):
    flags = torch.zeros(M, dtype=torch.bool, device=DEV)
    flags[so[(so >= 0) & (so < M)].long()] = True
    return flags


def poison(like):
    """Leaves NaN in the memory that the next tensor of this size is given."""
    torch.full_like(like, float("nan"))


# rows that get zeros beforehand, and rows that are found among the pairs (1024 bytes and 32 MB or more)
@pytest.mark.parametrize("T,k,H,extra,dtype", [
    (4, 2, 64, 0, BF16), (33, 8, 264, 0, F32), (33, 8, 264, 5, BF16), (1, 1, 8, 0, BF16), (4097, 8, 512, 0, BF16),
    (2100, 8, 1024, 0, BF16), (2100, 8, 1024, 3, BF16), (701, 6, 2056, 0, F32), (1, 64, 131072 * 4, 0, BF16)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_rows_of_a_new_dy(P, T, k, H, extra, dtype, drop):
    M = T * k + extra
    g = torch.Generator(device=DEV).manual_seed(T + H)
    y = torch.randn((M, H), generator=g, device=DEV).to(dtype)
    dout = torch.randn((T, H), generator=g, device=DEV).to(dtype)
    gates = torch.rand((T, k), generator=g, device=DEV)
    so = slots(T, k, M, T + k, drop)
    on = named(so, M)
    for want_dgates in (True, False):
        want, _ = P.moe_combine_rows_bwd(dout, y, so, gates, want_dgates=want_dgates, dy=torch.zeros_like(y))
        poison(y)
        got, _ = P.moe_combine_rows_bwd(dout, y, so, gates, want_dgates=want_dgates)
        assert torch.equal(got, want) and (got[~on] == 0).all()
    # slot_of in one row, as the router gives it
    poison(y)
    assert torch.equal(P.moe_combine_rows_bwd(dout, y, so.view(-1), gates)[0], want)


def test_no_tokens(P):
    y = torch.ones((20000, 1024), dtype=BF16, device=DEV)
    poison(y)
    dy, _ = P.moe_combine_rows_bwd(y[:0], y, torch.zeros((0, 3), dtype=torch.int32, device=DEV))
    assert (dy == 0).all()


# one row and odd counts, rows around the workgroups' shares (multiples of 32 a workgroup), pairs around the loads' batches
@pytest.mark.parametrize("M,H,pairs", [(1, 8, 1), (31, 8, 5), (257, 72, 300), (8192, 8, 4095), (8193, 16, 32768), (70001, 24, 32773),
                                       (70001, 8, 200001), (3, 65536, 4)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zero_unnamed(P, M, H, pairs, dtype):
    g = torch.Generator().manual_seed(M + pairs)
    # slots outside, and slots that stand several times
    so = torch.randint(-M // 8 - 1, M + M // 8 + 1, (pairs + 1,), generator=g).to(torch.int32).to(DEV)
    so[pairs // 2] = -2 ** 31
    for s in (so[:pairs], so[1:]):                    # 16-byte aligned and not
        buf = torch.full(((M + 2) * H,), 3.0, dtype=dtype, device=DEV)
        x = buf[H:-H].view(M, H)
        x.copy_(torch.randn((M, H), generator=torch.Generator().manual_seed(1)))
        want = x * named(s, M)[:, None]
        got = P.moe_rows_zero_unnamed(x, s.view(-1, 1))
        assert got is x and torch.equal(x, want)
        assert (buf[:H] == 3.0).all() and (buf[-H:] == 3.0).all()


def test_more_rows_than_the_workgroups_bits(P):
    """Rows past 256 workgroups of 2^18, and past 2^32 bytes."""
    M, H = (1 << 26) + 1000, 64
    x = torch.ones((M, H), dtype=BF16, device=DEV)
    so = torch.tensor([[0, M - 1, 1 << 18, (1 << 26) + 5, 12345678]], dtype=torch.int32, device=DEV)
    P.moe_rows_zero_unnamed(x, so)
    assert (x[so[0].long()] == 1).all() and int((x[:, 0] != 0).sum()) == 5 and int((x[:, 63] != 0).sum()) == 5


def test_streams_and_replayed_graph(P):
    T, k, H = 2100, 8, 1024
    M = T * k
    y, dout = torch.randn((M, H), device=DEV).to(BF16), torch.randn((T, H), device=DEV).to(BF16)
    so = slots(T, k, M, 0, 0.3)
    run = lambda: P.moe_combine_rows_bwd(dout, y, so, want_dgates=False)[0]  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for r in range(3):
        so.copy_(slots(T, k, M, 10 + r, 0.2))
        held.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(run(), held), r
