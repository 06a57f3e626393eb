"""adamw_step against fp64, and its 8-bit states against the oracle's random numbers.

Tolerances, with u = 2^-24. m and v are products and a sum, each rounded: off by at most 4 u of the sum of
their terms' magnitudes. The update's root, quotient, products and its rounded scalars stay within
16 u of it, and m's error passes through it: |p - ref| <= 2 u |p| + lr (16 u |upd| + E_m / d) where
d is the denominator. States in 8 bits: a value lies between two neighbours of the E4M3 grid of its
block, and goes up when the 16-bit random value is below floor(2^16 f), f its place between them.
The kernel's f is off by at most 16 * 4 u (16 steps of the grid an octave), below 2^-18: only where
r16 is within 1.5 of 2^16 f may the choice be the other one.
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
HY = dict(beta1=0.9, beta2=0.95, eps=1e-8)


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


def decode(codes, e8m0, n):
    v = codes.cpu().view(torch.float8_e4m3fn).double()
    return v * torch.exp2(e8m0.cpu().double() - 127).repeat_interleave(32)[:n]


def make(P, lens, bits, gdt, seed, copy=True, moments=True):
    g = torch.Generator().manual_seed(seed)
    ts = []
    for i, n in enumerate(lens):
        p = torch.randn(n, generator=g) * 0.02
        grad = (torch.randn(n, generator=g) * 10.0 ** (-1 - i % 4)).to(gdt)
        t = P.AdamWTensor.new(p.to(DEV), grad.to(DEV), bits, torch.full((n,), 5.0, dtype=torch.bfloat16, device=DEV) if copy else None,
                              weight_decay=0.1 if i % 2 else 0.0)
        if moments and bits == 32:
            t.m.copy_(torch.randn(n, generator=g) * 10.0 ** (-2 - i % 4))
            t.v.copy_((torch.randn(n, generator=g) * 10.0 ** (-1 - i % 4)) ** 2)
        elif moments:
            t.m.copy_(torch.randint(0, 256, (n,), generator=g).to(torch.uint8))
            t.m[(t.m & 127) == 127] = 3
            t.v.copy_(torch.randint(1, 127, (n,), generator=g).to(torch.uint8))
            t.m_e8m0.copy_(torch.randint(108, 112, t.m_e8m0.shape, generator=g).to(torch.uint8))
            t.v_e8m0.copy_(torch.randint(110, 114, t.v_e8m0.shape, generator=g).to(torch.uint8))
        ts.append(t)
    return ts


def state(t, bits):
    n = t.param.numel()
    if bits == 32:
        return t.m.double().cpu(), t.v.double().cpu()
    return decode(t.m, t.m_e8m0, n), decode(t.v, t.v_e8m0, n) ** 2


def reference(t, bits, lr, step, gs=1.0, beta1=0.9, beta2=0.95, eps=1e-8):
    g = t.grad.double().cpu() * gs
    m0, v0 = state(t, bits)
    m, v = beta1 * m0 + (1 - beta1) * g, beta2 * v0 + (1 - beta2) * g * g
    em = 4 * U * (beta1 * m0.abs() + (1 - beta1) * g.abs())
    d = torch.sqrt(v / (1 - beta2 ** step)) + eps
    upd = m / (1 - beta1 ** step) / d
    p0 = t.param.double().cpu()
    p = p0 * (1 - lr * t.weight_decay) - lr * upd
    pb = 2 * U * p0.abs() + U * p.abs() + lr * (16 * U * upd.abs() + em / (1 - beta1 ** step) / d)
    return p, pb, m, em, v, 4 * U * v


def within(got, ref, bound, what):
    bad = ~((got.double().cpu() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values outside the bound, first at {bad.nonzero()[0].tolist()}"


LENS = [1, 7, 8, 31, 32, 33, 2047, 2048, 2049, 5000, 12345, 3, 64, 100000]


def exponent(amax):
    """Smallest e in [-127, 127] with amax <= 448 2^e."""
    e = np.full(amax.shape, -127)
    nz = amax > 0
    e[nz] = np.clip(np.ceil(np.log2(amax[nz] / 448.0)), -127, 127)
    e = np.where(amax > 448.0 * 2.0 ** e, e + 1, e)
    return np.where((e > -127) & (amax <= 448.0 * 2.0 ** (e - 1.0)), e - 1, e)


def check_sr(codes, e8m0, value, seed, stream, positive, what, first=0):
    """The stored codes are the stochastic rounding of `value`, values `first` .. of a tensor, under
    (seed, stream)."""
    n = value.numel()
    val = np.zeros((n + 31) // 32 * 32)
    val[:n] = value.numpy()
    blocks = val.reshape(-1, 32)
    e = e8m0.cpu().numpy().astype(int) - 127
    want = exponent(np.abs(blocks).max(1))
    off = e != want
    amax = np.abs(blocks).max(1)[off]
    near = np.minimum(np.abs(amax / (448.0 * 2.0 ** want[off]) - 1), np.abs(amax / (448.0 * 2.0 ** (want[off] - 1.0)) - 1))
    assert (near <= 8 * U).all(), f"{what}: a block's scale"
    got = decode(codes, e8m0, n).numpy()
    scale = np.repeat(2.0 ** e.astype(float), 32)[:n]
    y = np.abs(val[:n]) / scale
    step = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    lo = np.floor(y / step) * step
    f = (y - lo) / step
    r16 = O.rand16_array(seed, stream, first + np.arange(n)).astype(np.float64)
    up = r16 < np.floor(f * 65536.0)
    expect = lo + step * up
    if positive:
        expect = np.where((y > 0) & (expect == 0), 2.0 ** -9, expect)
    # a value on a grid point may be read from either side of it, by an error far below a step
    edge = np.minimum(f, 1 - f) < 1e-5
    wrong = np.abs(got) / scale != expect
    allowed = (np.abs(f * 65536.0 - r16) <= 1.5) | edge
    assert not (wrong & ~allowed).any(), f"{what}: {(wrong & ~allowed).sum()} codes"
    assert (np.abs(np.abs(got) / scale - y)[~edge] <= step[~edge]).all(), what
    sg = np.sign(val[:n]) * np.sign(got)
    assert (sg >= 0).all(), f"{what}: signs"


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
def test_step(P, bits, gdt):
    """Lengths around the block, the piece and the chunk of a workgroup; every second tensor decays."""
    ts = make(P, LENS, bits, gdt, 3)
    refs = [reference(t, bits, 1e-2, 7) for t in ts]
    grads = [t.grad.clone() for t in ts]
    P.adamw_step(P.AdamWPlan(ts), lr=1e-2, step=7, seed=11, rng_stream=5, **HY)
    torch.cuda.synchronize()
    for i, (t, (p, pb, m, em, v, ev)) in enumerate(zip(ts, refs)):
        within(t.param, p, pb, f"p {i}")
        assert torch.equal(t.copy, t.param.to(torch.bfloat16)) and torch.equal(t.grad, grads[i])
        if bits == 32:
            within(t.m, m, em, f"m {i}")
            within(t.v, v, ev, f"v {i}")
        elif t.param.numel() <= 12345:
            check_sr(t.m, t.m_e8m0, m, 11 + 7, 5 + 2 * i, False, f"m {i}")
            check_sr(t.v, t.v_e8m0, v.sqrt(), 11 + 7, 5 + 2 * i + 1, True, f"v {i}")


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_equal_one_by_one(P, bits):
    """400 tensors in one call and the same tensors each in a call of its own: the same bits (in 8 bits
    with the stream that the list gives each)."""
    lens = [1 + (i * 37) % 900 for i in range(400)]
    a, b = make(P, lens, bits, torch.float32, 9), make(P, lens, bits, torch.float32, 9)
    P.adamw_step(P.AdamWPlan(a), lr=1e-3, step=3, seed=2, rng_stream=8, **HY)
    for i, t in enumerate(b):
        P.adamw_step(P.AdamWPlan([t]), lr=1e-3, step=3, seed=2, rng_stream=8 + 2 * i, **HY)
    for s, t in zip(a, b):
        for k in ("param", "m", "v", "copy", "m_e8m0", "v_e8m0"):
            u, w = getattr(s, k), getattr(t, k)
            assert u is None or torch.equal(u, w), k


@pytest.mark.parametrize("bits", [32, 8])
def test_neighbouring_memory_is_left_alone(P, bits):
    """Tensors that end inside a block and a chunk, in larger buffers of known bytes."""
    n = 2048 + 41
    raw = {k: torch.full((n + 64,), 77, dtype=torch.uint8 if bits == 8 else torch.float32, device=DEV) for k in "mv"}
    e8 = {k: torch.full(((n + 31) // 32 + 32,), 99, dtype=torch.uint8, device=DEV) for k in "mv"}
    p = torch.full((n + 64,), 2.0, device=DEV)
    cp = torch.full((n + 64,), 2.0, dtype=torch.bfloat16, device=DEV)
    g = torch.randn(n, device=DEV)
    for k in "mv":
        raw[k][16:16 + n] = 0
        e8[k][16:-16] = 0
    kw = dict(m_e8m0=e8["m"][16:-16], v_e8m0=e8["v"][16:-16]) if bits == 8 else {}
    t = P.AdamWTensor(p[16:16 + n], g, raw["m"][16:16 + n], raw["v"][16:16 + n], cp[16:16 + n], **kw)
    P.adamw_step(P.AdamWPlan([t]), lr=1e-2, step=1, **HY)
    for buf, c in ((raw["m"], 77), (raw["v"], 77), (p, 2), (cp, 2)):
        assert (buf[:16] == c).all() and (buf[16 + n:] == c).all()
    for k in "mv":
        assert (e8[k][:16] == 99).all() and (e8[k][-16:] == 99).all()


def test_first_steps_from_zero_moments(P):
    """From zero moments, by both widths: the first step moves every weight by lr times the sign of its
    gradient (m / (1 - b1) = g, sqrt(v / (1 - b2)) = |g|); 16 u of it, and eps / |g|."""
    for bits in (32, 8):
        ts = make(P, [4097], bits, torch.float32, 4, copy=False, moments=False)
        p0, g = ts[0].param.double().cpu(), ts[0].grad.double().cpu()
        P.adamw_step(P.AdamWPlan(ts), lr=1e-2, step=1, **HY)
        ref = p0 - 1e-2 * g / (g.abs() + 1e-8)
        within(ts[0].param, ref, 3 * U * p0.abs() + 1e-2 * 24 * U, f"p {bits}")


def test_slow_decay_survives_8_bits(P):
    """With zero gradients sqrt(v) shrinks by sqrt(b2) a step, far below half a step of E4M3; stochastic
    rounding keeps its mean. Each step adds at most half a code step (1/16 of the value) of deviation, so
    50 steps at most 0.45 a value and 0.45 / 256 over 65536 of them; five of those are 0.009."""
    n, steps, b2 = 65536, 50, 0.999
    t = P.AdamWTensor.new(torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), 8)
    t.v.copy_(torch.randint(0x60, 0x7E, (n,), dtype=torch.uint8))
    t.v_e8m0.fill_(120)
    s0 = decode(t.v, t.v_e8m0, n)
    plan = P.AdamWPlan([t])
    for k in range(steps):
        P.adamw_step(plan, lr=0.0, step=1 + k, beta1=0.9, beta2=b2, seed=3)
    ratio = float(decode(t.v, t.v_e8m0, n).sum() / s0.sum())
    assert abs(ratio - b2 ** (steps / 2)) < 0.009 * b2 ** (steps / 2)


def test_scalars_on_the_device_and_graph(P):
    """lr, step and grad_scale on the device give the bits of the host's scalars (a power of two scales
    exactly), eager and in a graph that is replayed with the step counted between the replays."""
    lens = [100, 5000, 33]
    for bits in (32, 8):
        a, b, c = (make(P, lens, bits, torch.float32, 6) for _ in range(3))
        for t in b + c:
            t.grad.mul_(4.0)
        pa, pb, pc = P.AdamWPlan(a), P.AdamWPlan(b), P.AdamWPlan(c)
        lr = torch.tensor(1e-3, device=DEV)
        gs = torch.tensor([0.25], device=DEV)
        sb, sc = (torch.tensor([2], dtype=torch.int64, device=DEV) for _ in range(2))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            P.adamw_step(pc, lr=lr, step=sc, grad_scale=gs, seed=9, **HY)
        for k in range(3):
            P.adamw_step(pa, lr=float(np.float32(1e-3)), step=2 + k, seed=9, **HY)
            P.adamw_step(pb, lr=lr, step=sb, grad_scale=gs, seed=9, **HY)
            graph.replay()
            torch.cuda.synchronize()
            for x, y, z in zip(a, b, c):
                for f in ("param", "m", "v", "copy"):
                    assert torch.equal(getattr(x, f), getattr(y, f)), (bits, k, f)
                    assert torch.equal(getattr(x, f), getattr(z, f)), (bits, k, f)
            sb += 1
            sc += 1


def test_not_finite_gradients_stay_in_their_value(P):
    for bits in (32, 8):
        a, b = make(P, [300], bits, torch.float32, 6), make(P, [300], bits, torch.float32, 6)
        b[0].grad[100] = float("nan")
        for ts in (a, b):
            P.adamw_step(P.AdamWPlan(ts), lr=1e-3, step=2, **HY)
        keep = torch.arange(300, device=DEV) != 100
        assert torch.isnan(b[0].param[100]) and torch.equal(a[0].param[keep], b[0].param[keep])


def test_another_states_table_is_left_alone(P):
    """A table built for states of one width, run as the other: nothing is written."""
    ts = make(P, [5000], 32, torch.float32, 2)
    plan = P.AdamWPlan(ts)
    before = [ts[0].param.clone(), ts[0].m.clone(), ts[0].v.clone()]
    plan.state_bits = 8
    P.adamw_step(plan, lr=1.0, step=1, **HY)
    plan.state_bits, plan.chunks = 32, plan.chunks + 5
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (ts[0].param, ts[0].m, ts[0].v)))
    P.adamw_step(plan, lr=1e-2, step=1, **HY)   # chunks past the table's are skipped
    assert not torch.equal(before[0], ts[0].param) and torch.isfinite(ts[0].param).all()


def test_empty_tensors_take_no_part(P):
    """Tensors of no values beside others: the others' step is the one without them (each keeps its place
    in the list, and with it its stream of random numbers)."""
    for bits in (32, 8):
        a, b = make(P, [100, 70], bits, torch.float32, 6), make(P, [100, 70], bits, torch.float32, 6)
        none = P.AdamWTensor.new(torch.empty(0, device=DEV), torch.empty(0, device=DEV), bits)
        P.adamw_step(P.AdamWPlan([a[0], a[1], none]), lr=1e-3, step=2, seed=4, **HY)
        P.adamw_step(P.AdamWPlan(b), lr=1e-3, step=2, seed=4, **HY)
        for s, t in zip(a, b):
            assert torch.equal(s.param, t.param) and torch.equal(s.m, t.m) and torch.equal(s.v, t.v)
        P.adamw_step(P.AdamWPlan([none]), lr=1e-3, step=2, **HY)


def test_offsets_past_32_bits(P):
    """A tensor of 2^31 + 5000 values (states in 8 bits, bf16 gradient): its last values against the same
    values as a tensor of their own, with the random numbers of their indices through check_sr."""
    n = (1 << 31) + 5000
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    tail = 4096
    gen = torch.Generator().manual_seed(3)
    p[-tail:] = torch.randn(tail, generator=gen).to(DEV) * 0.02
    g[-tail:] = (torch.randn(tail, generator=gen) * 1e-2).to(torch.bfloat16).to(DEV)
    t = P.AdamWTensor.new(p, g, 8)
    small = P.AdamWTensor.new(p[-tail:].clone(), g[-tail:].clone(), 32)
    refs = reference(small, 32, 1e-2, 1)
    P.adamw_step(P.AdamWPlan([t]), lr=1e-2, step=1, seed=3, **HY)
    within(t.param[-tail:], refs[0], refs[1], "p")
    assert (t.param[:1000] == 0).all() and (t.param[(1 << 31):(1 << 31) + 100] == 0).all()
    # the last whole blocks: the tail begins inside one, 5000 - 4096 = 904 = 28 * 32 + 8
    at = n - tail + 24
    assert at % 32 == 0
    m, v = refs[2][24:], refs[4][24:]
    check_sr(t.m[at:], t.m_e8m0[at // 32:], m, 3 + 1, 0, False, "m", first=at)
    check_sr(t.v[at:], t.v_e8m0[at // 32:], v.sqrt(), 3 + 1, 1, True, "v", first=at)
