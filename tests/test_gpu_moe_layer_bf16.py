"""The expert layer on unquantized activations as it is used: a training step in bf16 (route, w1 and w3 with SwiGLU,
w2, the gates' sum, and the gradients of the input, both weights and the gates) against autograd in fp64, and a
decoded token's layer with NVFP4 weights against fp64.

The bounds here are coarse on purpose (each call has its own bounds in its own file): every intermediate that is
rounded to bf16 carries 2^-8 of itself, so a result of three roundings in a row stays within 4 * 2^-8 of the fp64
result in norm, whatever the cancellation inside a single value."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def mk(shape, std, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(DEV)


def near(got, ref, what, bound=4 * 2.0 ** -8):
    err = float((got.double() - ref).norm() / ref.norm())
    assert err <= bound, f"{what}: {err:.2e} off"


def experts(x, w13, w2, ids, E, F):
    """fp64 rows [T, k, H] of each token's experts."""
    T, k = ids.shape
    H = w2.shape[1] if w2.dim() == 3 else w2.shape[0] // E
    y = torch.zeros((T, k, H), dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        h = x[t] @ w13[e].t()
        a = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
        y = y.index_put((t, j), a @ w2[e].t())
    return y


@pytest.mark.parametrize("T,E,k,H,F", [(70, 6, 2, 264, 136), (900, 4, 3, 512, 264), (5, 12, 4, 128, 64)])
def test_training_step(P, T, E, k, H, F):
    x, shared, dout = mk((T, H), 1.0, 1), mk((T, H), 0.5, 2), mk((T, H), 1.0, 3)
    w13, w2 = mk((E * 2 * F, H), 1.2 / H ** 0.5, 4), mk((E * H, F), F ** -0.5, 5)
    g = torch.Generator().manual_seed(6)
    logits = torch.randn((T, E), generator=g).to(DEV)
    M = T * k
    r = P.moe_route_topk(logits, k)
    off, gather = r["offsets"], r["gather"]
    slot_of, gates = r["slot_of"], r["gates"]
    a, h13 = P.moe_grouped_gemm_fwd_bf16(x, w13, off, M, 2 * F, P.EPI_SWIGLU, gather=gather, save_h13=True)
    y = P.moe_grouped_gemm_fwd_bf16(a, w2, off, M, H)
    out = P.moe_combine_rows_fwd(y, slot_of, gates, add=shared)
    dy, dgates = P.moe_combine_rows_bwd(dout, y, slot_of, gates)
    dh13, dw2 = P.moe_grouped_gemm_bwd_bf16(dy, None, w2, off, M, H, h13=h13)
    da, dw13 = P.moe_grouped_gemm_bwd_bf16(dh13, x, w13, off, M, 2 * F, gather=gather, da_dtype=torch.float32)
    dx = P.moe_combine_rows_fwd(da, slot_of.view(T, k))

    X, W13, W2 = (t.double().requires_grad_() for t in (x, w13, w2))
    G = gates.double().requires_grad_()
    Y = experts(X, W13.view(E, 2 * F, H), W2.view(E, H, F), r["ids"], E, F)
    OUT = (Y * G[:, :, None]).sum(1) + shared.double()
    OUT.backward(dout.double())
    for name, got, ref in (("out", out, OUT.detach()), ("dx", dx, X.grad), ("dw13", dw13, W13.grad), ("dw2", dw2, W2.grad),
                           ("dgates", dgates, G.grad)):
        near(got, ref, name)


@pytest.mark.parametrize("T", [1, 3, 16, 40])
def test_decoded_tokens(P, T):
    """Two calls a layer: w1 and w3 with SwiGLU, then w2 with the gates' sum and the shared expert's row."""
    E, k, H, F = 12, 4, 512, 320
    w13 = P.nvfp4_quantize(mk((E * 2 * F, H), 1.2 / H ** 0.5, 11), P.NVFP4_WEIGHT, rows_per_outer=F)
    w2 = P.nvfp4_quantize(mk((E * H, F), F ** -0.5, 12), P.NVFP4_WEIGHT, rows_per_outer=H)
    x, shared = mk((T, H), 1.0, 13), mk((T, H), 0.5, 14)
    g = torch.Generator().manual_seed(15)
    r = P.moe_route_topk(torch.randn((T, E), generator=g).to(DEV), k)
    a = P.moe_gemv_nvfp4(x, w13, 2 * F, r["ids"], P.EPI_SWIGLU)
    out = P.moe_gemv_nvfp4(a, w2, H, r["ids"], gates=r["gates"], add=shared)

    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    grid = torch.cat([grid, -grid])

    def value(q):
        c = q.codes.long()
        v = torch.stack([grid[c % 16], grid[c // 16]], 2).flatten(1)
        return v * q.scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) \
            * q.outer.double().repeat_interleave(q.rows_per_outer)[:, None]

    Y = experts(x.double(), value(w13).view(E, 2 * F, H), value(w2).view(E, H, F), r["ids"], E, F)
    near(out, (Y * r["gates"].double()[:, :, None]).sum(1) + shared.double(), "out")
    # the same layer row by row: the pairs' rows, then the sum
    rows = P.moe_gemv_nvfp4(a, w2, H, r["ids"], P.EPI_F32)
    pair = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    near(P.moe_combine_rows_fwd(rows.view(T * k, H), pair, r["gates"], add=shared), out.double(), "row by row", 2.0 ** -8)


def test_quantized_backward_joins_a_tokens_slots(P):
    """The fp32 slot gradients of the quantized backward, added per token."""
    T, E, k, N, K = 60, 4, 2, 128, 96
    r = P.moe_route_topk(torch.randn((T, E), generator=torch.Generator().manual_seed(1)).to(DEV), k)
    xq = P.nvfp4_quantize(mk((T, K), 1.0, 2), P.NVFP4_ACT)
    wq = P.nvfp4_quantize(mk((E * N, K), 0.1, 3), P.NVFP4_WEIGHT, rows_per_outer=N)
    da, _, _ = P.moe_grouped_gemm_bwd(mk((T * k, N), 1.0, 4), xq, wq, r["offsets"], T * k, N, flags=P.BWD_DGRAD,
                                      gather=r["gather"])
    dx = P.moe_combine_rows_fwd(da, r["slot_of"].view(T, k), out_dtype=torch.float32)
    want = torch.zeros((T, K), dtype=torch.float64, device=DEV).index_add_(0, r["gather"].long(), da.double())
    # k terms in fp32
    assert ((dx.double() - want).abs() <= 4 * 2.0 ** -24 * da.double().abs().max() * k).all()
