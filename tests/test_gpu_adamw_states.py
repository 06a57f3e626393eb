"""The 8-bit states of adamw_step where their format ends: values that are not finite beside others in
a block, and values that lie on the grid under every exponent of a scale.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
HY = dict(beta1=0.9, beta2=0.95, eps=1e-8)


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


N, AT = 289, [5, 100, 101, 288]   # alone in a block, two beside each other, the only value of the last block


@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), 1e30, -3e38])
def test_a_value_past_the_range_leaves_its_block_alone(P, value, gdt):
    """Infinite and NaN gradients, and finite ones whose squares are past fp32: over three steps the other
    values of their blocks keep the weights, codes and scales of a twin that has zeros there; the value's
    own moments are NaN, and its weight with them from the next step on (a finite gradient's first step is
    the formula's m / inf)."""
    n = N
    g = torch.Generator().manual_seed(8)
    grads = [(torch.randn(n, generator=g) * 1e-2) for _ in range(3)]
    for k in grads:
        k[AT] = 0.0
    start = torch.randn(n, generator=g) * 0.02
    codes = torch.randint(1, 127, (2, n), generator=g).to(torch.uint8)
    codes[:, AT] = 0
    keep = torch.ones(n, dtype=torch.bool)
    keep[AT] = False
    ts = []
    for _ in range(2):
        t = P.AdamWTensor.new(start.to(DEV), torch.zeros(n, dtype=gdt, device=DEV), 8,
                              torch.zeros(n, dtype=torch.bfloat16, device=DEV), 0.1)
        t.m.copy_(codes[0])
        t.v.copy_(codes[1])
        t.m_e8m0.fill_(110)
        t.v_e8m0.fill_(112)
        ts.append(t)
    a, b = ts
    pa, pb = P.AdamWPlan([a]), P.AdamWPlan([b])
    for step in range(1, 4):
        a.grad.copy_(grads[step - 1])
        b.grad.copy_(grads[step - 1])
        if step == 1:
            b.grad[AT] = value
        for plan in (pa, pb):
            P.adamw_step(plan, lr=1e-3, step=step, seed=5, rng_stream=3, **HY)
        for k in ("param", "copy", "m", "v"):
            assert torch.equal(getattr(a, k)[keep], getattr(b, k)[keep]), (step, k)
        assert torch.equal(a.m_e8m0, b.m_e8m0) and torch.equal(a.v_e8m0, b.v_e8m0), step
        for k in ("m", "v"):
            assert torch.isnan(getattr(b, k).view(torch.float8_e4m3fn).float()[AT]).all(), (step, k)
        if step > 1 or not np.isfinite(value):
            assert torch.isnan(b.param[AT]).all()
        else:
            assert torch.equal(b.param[AT], a.param[AT])


def test_every_exponent_of_a_scale(P):
    """Moments that a step leaves as they are (no gradient, betas that are 1 in fp32), under each exponent
    that the moments reach (of m all from 2^-127 on to fp32's end, of sqrt(v) those whose squares are
    normal), 131072 values an exponent with a block's largest at 448 2^e. The scale's reciprocal is 2^-e or
    one ulp below it, never above: no code becomes NaN or grows, none loses more than one step of the grid,
    and that where the random number is 65535 alone, 2 of 131072 expected and 17 hardly ever (1e-10)."""
    per = 1 << 12   # blocks of an exponent
    for lo, hi, which in ((-127, 119, "m"), (-50, 54, "v")):
        e = torch.arange(lo, hi + 1, device=DEV).repeat_interleave(per)
        g = torch.Generator(device=DEV).manual_seed(2)
        codes = torch.randint(1, 0x7F, (e.numel(), 32), generator=g, device=DEV)
        codes[:, 0] = 0x7E
        if which == "m":
            codes |= torch.randint(0, 2, codes.shape, generator=g, device=DEV) << 7
        codes, scales = codes.to(torch.uint8).view(-1), (e + 127).to(torch.uint8)
        n = codes.numel()
        t = P.AdamWTensor.new(torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), 8)
        getattr(t, which).copy_(codes)
        getattr(t, which + "_e8m0").copy_(scales)
        plan = P.AdamWPlan([t])
        for step in range(1, 4):
            P.adamw_step(plan, lr=0.0, step=step, beta1=1 - 2.0 ** -30, beta2=1 - 2.0 ** -30, seed=1)
            assert torch.equal(getattr(t, which + "_e8m0"), scales), (which, step)
            lost = codes.int() - getattr(t, which).int()
            assert ((lost == 0) | (lost == 1)).all(), (which, step)
            count = lost.view(-1, per * 32).sum(1)
            assert (count < 17).all(), f"{which}: {count.max()} at exponent {int(count.argmax()) + lo}"
            codes = getattr(t, which).clone()
