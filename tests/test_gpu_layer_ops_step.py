"""One training step of a layer's dense side around the routed experts, as a program runs it: the
residual norm, the routed experts through the library's existing calls (NVFP4 forward, RHT32 + S2F6
payload, combine), the shared expert with the routed sum added in its epilogue, the backward of the
dense side, one AdamW step over its weights and the requantization of the updated expert weights.

The dense side is checked against fp64 with each stage's own inputs (the earlier stages' outputs), at
the bounds of the single operators' tests: a chain of stages then holds if each stage holds. The
composed gradient is checked against fp64 end to end as well: every stage rounds to bf16 once or
twice (2^-8 each), and the relative Frobenius error of a chain of n such independent roundings stays
below n 2^-8; five stages (y, a and h13, dy, dh13, dx) bound it by 5 * 2 * 2^-8 = 0.04.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
T, H, F, E, K = 200, 256, 128, 8, 2
U, B = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def setup(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    return dict(x=r(T, H).to(torch.bfloat16), res=r(T, H).float(), gamma=(1 + 0.1 * r(H)).float(),
                logits=r(T, E).float(), ew13=r(E * 2 * F, H, std=0.05).float(), ew2=r(E * H, F, std=0.05).float(),
                w13=r(2 * F, H, std=0.07).float(), w2=r(H, F, std=0.09).float(),
                dout=r(T, H, std=0.1).to(torch.bfloat16), dz_later=r(T, H, std=0.1).float())


def forward(P, d, w13, w2, ew13q, ew2q):
    n = P.rmsnorm_residual_fwd(d["x"], d["gamma"], residual=d["res"], want_mxfp8=True, want_rstd=True)
    rt = P.moe_route_topk(d["logits"], K)
    M = T * K
    xq = P.nvfp4_quantize(n.y, P.NVFP4_ACT)
    act, _ = P.moe_grouped_gemm_fwd(xq, ew13q, rt["offsets"], M, 2 * F, P.EPI_SWIGLU, gather=rt["gather"])
    aq = P.nvfp4_quantize(act, P.NVFP4_ACT)
    codes, e8 = P.moe_grouped_gemm_fwd(aq, ew2q, rt["offsets"], M, H, P.EPI_RHT32_S2F6, rht_sign_mask=0x5A5A1234)
    routed = P.moe_combine_s2f6(codes, e8, 0x5A5A1234, rt["slot_of"], rt["gates"])
    out, h13 = P.swiglu_ffn_fwd(n.y, w13, w2, add=routed, save_h13=True)
    return n, routed, out, h13


def quantize_experts(P, d):
    return (P.nvfp4_quantize(d["ew13"].to(torch.bfloat16), P.NVFP4_WEIGHT, rows_per_outer=2 * F),
            P.nvfp4_quantize(d["ew2"].to(torch.bfloat16), P.NVFP4_WEIGHT, rows_per_outer=H))


def rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


@pytest.mark.parametrize("bits", [32, 8])
def test_training_step_of_the_dense_side(P, bits):
    c = setup(11)
    d = {k: v.to(DEV) for k, v in c.items()}
    w13, w2 = d["w13"].to(torch.bfloat16), d["w2"].to(torch.bfloat16)
    n, routed, out, h13 = forward(P, d, w13, w2, *quantize_experts(P, d))
    # the norm's 8-bit output is the one of the quantizer within a rounding of y: bf16(y) against y
    q8, e8, _ = P.mxfp8_quantize(n.y)
    v8 = q8.view(torch.float8_e4m3fn).float() * torch.exp2(e8.float() - 127).repeat_interleave(32, 1)
    vn = n.codes.view(torch.float8_e4m3fn).float() * torch.exp2(n.e8m0.float() - 127).repeat_interleave(32, 1)
    y = n.y.float()
    scale = torch.exp2(torch.maximum(e8, n.e8m0).float() - 127).repeat_interleave(32, 1)
    assert ((v8 - vn).abs() <= (2 ** -4 * 2 + B * 2) * y.abs().clamp_min(2.0 ** -6 * scale)).all()

    # gradients: through the shared expert, then the norm (the routed experts' own input gradient is
    # the existing calls' and stays out of this chain)
    dy, dw13, dw2 = P.swiglu_ffn_bwd(d["dout"], n.y, w13, w2, h13)
    dz, dgamma = P.rmsnorm_residual_bwd(dy, n.z, d["gamma"], n.rstd, dres=d["dz_later"])

    ref = {k: c[k].double().requires_grad_() for k in ("x", "gamma")}
    ref["w13"], ref["w2"] = (w.double().cpu().requires_grad_() for w in (w13, w2))
    z = ref["x"] + c["res"].double()
    z.retain_grad()
    yr = z / torch.sqrt((z * z).mean(1, keepdim=True) + 1e-6) * ref["gamma"]
    hr = yr @ ref["w13"].t()
    outr = (hr[:, :F] * torch.sigmoid(hr[:, :F]) * hr[:, F:]) @ ref["w2"].t() + routed.double().cpu()
    ((outr * c["dout"].double()).sum() + (z * c["dz_later"].double()).sum()).backward()
    for got, want in ((n.y, yr), (out, outr), (dz, z.grad), (dgamma, ref["gamma"].grad), (dw13, ref["w13"].grad),
                      (dw2, ref["w2"].grad)):
        assert rel(got, want.detach()) <= 0.04

    # the update, and the experts' weights through the quantizer from the copies that it wrote
    params = {"gamma": (d["gamma"].clone(), dgamma), "w13": (d["w13"].clone(), dw13), "w2": (d["w2"].clone(), dw2),
              "ew13": (d["ew13"].clone(), torch.randn_like(d["ew13"]) * 1e-3)}
    copies = {k: torch.empty(p.numel(), dtype=torch.bfloat16, device=DEV) for k, (p, _) in params.items()}
    plan = P.AdamWPlan([P.AdamWTensor.new(p.view(-1), g.view(-1), bits, copies[k], 0.1 if k != "gamma" else 0.0)
                        for k, (p, g) in params.items()])
    before = {k: p.double().cpu().view(-1) for k, (p, _) in params.items()}
    P.adamw_step(plan, lr=1e-3, step=1, seed=5)
    for k, (p, g) in params.items():
        gd = g.double().cpu().view(-1)
        want = before[k] * (1 - 1e-3 * (0.1 if k != "gamma" else 0.0)) - 1e-3 * gd / (gd.abs() + 1e-8)
        err = (p.double().cpu().view(-1) - want).abs()
        assert (err <= 3 * U * before[k].abs() + 1e-3 * 24 * U).all(), k
        assert torch.equal(copies[k], p.view(-1).to(torch.bfloat16))
    q = P.nvfp4_quantize(copies["ew13"].view(E * 2 * F, H), P.NVFP4_WEIGHT, rows_per_outer=2 * F)
    again = P.nvfp4_quantize(params["ew13"][0].to(torch.bfloat16), P.NVFP4_WEIGHT, rows_per_outer=2 * F)
    assert torch.equal(q.codes, again.codes) and torch.equal(q.outer, again.outer)


def test_step_in_a_graph(P):
    """The whole chain captured once, with its step count on the device, and replayed between eager steps
    of a twin: the same weights after each."""
    c = setup(12)
    d = {k: v.to(DEV) for k, v in c.items()}
    ew = quantize_experts(P, d)

    def program():
        master = {"w13": d["w13"].clone(), "w2": d["w2"].clone(), "gamma": d["gamma"].clone()}
        w = {k: torch.empty_like(master[k], dtype=torch.bfloat16) for k in ("w13", "w2")}
        grads = {k: torch.zeros_like(v) for k, v in master.items()}
        for k in w:
            w[k].copy_(master[k])
        plan = P.AdamWPlan([P.AdamWTensor.new(master[k].view(-1), grads[k].view(-1), 8,
                                              w[k].view(-1) if k in w else None) for k in master])
        count = torch.ones(1, dtype=torch.int64, device=DEV)
        x = dict(d, gamma=master["gamma"])

        def step():
            n, _, out, h13 = forward(P, x, w["w13"], w["w2"], *ew)
            dy, _, _ = P.swiglu_ffn_bwd(out, n.y, w["w13"], w["w2"], h13, dw13=grads["w13"], dw2=grads["w2"])
            _, dg = P.rmsnorm_residual_bwd(dy, n.z, master["gamma"], n.rstd)
            grads["gamma"].copy_(dg)
            P.adamw_step(plan, lr=1e-3, step=count, seed=3)
            count.add_(1)
        return step, master

    eager, me = program()
    captured, mg = program()
    keep = {k: v.clone() for k, v in mg.items()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured()
    assert all(torch.equal(mg[k], keep[k]) for k in mg)   # capturing ran nothing
    for k in range(3):
        eager()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(me[n], mg[n]) for n in me), f"replay {k}"
