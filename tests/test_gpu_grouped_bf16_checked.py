"""The grouped bf16 products with CHECK_INDICES: what breaks the contract is refused before the launch, what the products
do not read is not looked at."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
M, G, N, K, ROWS = 12, 2, 32, 40, 5


@pytest.fixture
def P(monkeypatch):
    import precision_moe_numerics_amd as P
    monkeypatch.setattr(P, "CHECK_INDICES", True)
    return P


def operands():
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    gather = torch.randint(0, ROWS, (M,), generator=g).to(torch.int32).to(DEV)
    return mk(ROWS, K), mk(G * N, K), mk(M, N), torch.tensor([0, 7, M], device=DEV), gather


def test_a_row_outside_is_refused(P):
    x, w, dy, off, gather = operands()
    P.moe_grouped_gemm_fwd_bf16(x, w, off, M, N, gather=gather)
    P.moe_grouped_gemm_bwd_bf16(dy, x, w, off, M, N, gather=gather)
    bad = gather.clone()
    bad[3] = ROWS
    with pytest.raises(P.PmnError):
        P.moe_grouped_gemm_fwd_bf16(x, w, off, M, N, gather=bad)
    with pytest.raises(P.PmnError):
        P.moe_grouped_gemm_bwd_bf16(dy, x, w, off, M, N, gather=bad)
    with pytest.raises(P.PmnError):
        P.moe_grouped_gemm_bwd_bf16(dy, x, w, off - 1, M, N, gather=gather)


def test_data_gradients_without_x(P):
    x, w, dy, off, gather = operands()
    want, _ = P.moe_grouped_gemm_bwd_bf16(dy, x, w, off, M, N, gather=gather)
    got, none = P.moe_grouped_gemm_bwd_bf16(dy, None, w, off, M, N, flags=P.BWD_DGRAD, gather=gather)
    assert none is None and torch.equal(got, want)
    with pytest.raises(P.PmnError):
        P.moe_grouped_gemm_bwd_bf16(dy, None, w, off - 1, M, N, flags=P.BWD_DGRAD, gather=gather)
