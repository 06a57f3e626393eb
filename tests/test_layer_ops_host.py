"""Refusals of the operators around the routed experts (norm, shared expert, AdamW), checked on the
host before anything is launched: through the C ABI with pointers that are never dereferenced, and
through the binding with tensors on the CPU."""
import ctypes as C

import pytest
import torch

import precision_moe_numerics_amd as P

FAKE, ODD = C.c_void_p(0x1000), C.c_void_p(0x1008)
EINVAL, ESHAPE, EALIGN, EWS = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    return P._lib


def test_norm_forward_refusals(lib):
    def f(x=FAKE, res=FAKE, rdt=0, gamma=FAKE, eps=1e-6, rows=4, cols=64, z=FAKE, y=FAKE, codes=FAKE, e=FAKE, rstd=FAKE):
        return lib.rmsnorm_residual_fwd(x, res, rdt, gamma, eps, rows, cols, z, y, codes, e, rstd, None)
    assert f(rdt=2) == EINVAL and f(eps=-1.0) == EINVAL and f(eps=float("nan")) == EINVAL
    assert f(cols=40) == ESHAPE and f(cols=36, codes=None, e=None) == ESHAPE and f(cols=0) == ESHAPE
    assert f(cols=32768 + 32) == ESHAPE and f(rows=-1) == ESHAPE and f(rows=1 << 31) == ESHAPE
    assert f(x=None) == EINVAL and f(gamma=None) == EINVAL and f(z=None) == EINVAL
    assert f(y=None, codes=None, e=None) == EINVAL and f(e=None) == EINVAL and f(codes=None) == EINVAL
    for k in ("x", "res", "gamma", "z", "y", "codes"):
        assert f(**{k: ODD}) == EALIGN, k
    assert f(rstd=C.c_void_p(0x1002)) == EALIGN
    assert f(rows=0, x=None, res=None, gamma=None) == 0


def test_norm_backward_refusals(lib):
    n = lib.rmsnorm_residual_bwd_workspace_size(4, 64)
    assert n > 0 and lib.rmsnorm_residual_bwd_workspace_size(4, 60) == 0

    def f(dy=FAKE, ddt=0, z=FAKE, zdt=1, gamma=FAKE, rstd=FAKE, dres=None, rows=4, cols=64, dz=FAKE, dg=FAKE, ws=FAKE, nb=n):
        return lib.rmsnorm_residual_bwd(dy, ddt, z, zdt, gamma, rstd, dres, rows, cols, dz, dg, ws, nb, None)
    assert f(ddt=3) == EINVAL and f(zdt=-1) == EINVAL and f(cols=60) == ESHAPE and f(rows=-2) == ESHAPE
    for k in ("dy", "z", "gamma", "rstd", "dz", "dg"):
        assert f(**{k: None}) == EINVAL, k
    assert f(ws=None) == EWS and f(nb=n - 1) == EWS
    for k in ("dy", "z", "gamma", "dres", "dz", "dg", "ws"):
        assert f(**{k: ODD}) == EALIGN, k
    assert f(rows=0, dg=None) == EINVAL


def test_ffn_refusals(lib):
    n = lib.swiglu_ffn_fwd_workspace_size(4, 64, 32)
    m = lib.swiglu_ffn_bwd_workspace_size(4, 64, 32)
    assert n >= 4 * 32 * 2 and m >= 4 * 32 * 6 and lib.swiglu_ffn_fwd_workspace_size(4, 60, 32) == 0

    def f(x=FAKE, w13=FAKE, w2=FAKE, add=None, M=4, H=64, F=32, h=None, y=FAKE, ws=FAKE, nb=n):
        return lib.swiglu_ffn_fwd(x, w13, w2, add, M, H, F, h, y, ws, nb, None)
    assert f(M=-1) == ESHAPE and f(H=60) == ESHAPE and f(F=36) == ESHAPE and f(H=0) == ESHAPE and f(F=0) == ESHAPE
    for k in ("x", "w13", "w2", "y"):
        assert f(**{k: None}) == EINVAL, k
    assert f(ws=None) == EWS and f(nb=n - 1) == EWS
    for k in ("x", "w13", "w2", "add", "h", "y", "ws"):
        assert f(**{k: ODD}) == EALIGN, k
    assert f(M=0, x=None, y=None, ws=None) == 0

    def b(dy=FAKE, x=FAKE, w13=FAKE, w2=FAKE, h=FAKE, M=4, H=64, F=32, flags=3, dx=FAKE, d13=FAKE, d2=FAKE, dt=0, ws=FAKE, nb=m):
        return lib.swiglu_ffn_bwd(dy, x, w13, w2, h, M, H, F, flags, dx, d13, d2, dt, ws, nb, None)
    assert b(flags=0) == EINVAL and b(flags=4) == EINVAL and b(flags=8 | 1) == EINVAL and b(dt=2) == EINVAL
    assert b(M=-1) == ESHAPE and b(H=4) == ESHAPE and b(F=12) == ESHAPE
    for k in ("dy", "x", "w13", "w2", "h", "dx", "d13", "d2"):
        assert b(**{k: None}) == EINVAL, k
    assert b(ws=None) == EWS and b(nb=m - 1) == EWS
    for k in ("dy", "x", "w13", "w2", "h", "dx", "d13", "d2", "ws"):
        assert b(**{k: ODD}) == EALIGN, k
    assert b(M=0, flags=1) == 0


def entry(**kw):
    d = dict(param=0x1000, grad=0x2000, copy=0x3000, m=0x4000, v=0x5000, m_e8m0=0x6000, v_e8m0=0x7000, n=100,
             weight_decay=0.0, grad_dtype=1)
    d.update(kw)
    return P._AdamWEntry(*(d[f[0]] for f in P._AdamWEntry._fields_))


def test_adamw_table_refusals(lib):
    def build(e, bits=8, short=0, count=1, misalign=0):
        arr = (P._AdamWEntry * 1)(e)
        size = lib.adamw_table_size(arr, 1)
        buf = (C.c_int64 * (size // 8 + 2))()
        chunks = C.c_int64(-7)
        st = lib.adamw_table_build(arr, count, bits, C.addressof(buf) + misalign, size - short, C.byref(chunks))
        return st, chunks.value
    assert build(entry()) == (0, 1) and build(entry(n=0, param=None)) == (0, 0)
    assert build(entry(), bits=16)[0] == EINVAL and build(entry(n=-1))[0] == ESHAPE
    assert build(entry(), count=-1)[0] == ESHAPE and build(entry(grad_dtype=2))[0] == EINVAL
    assert build(entry(n=(1 << 40) + 1))[0] == ESHAPE
    assert build(entry(n=1 << 35))[0] == ESHAPE   # 2^24 chunks
    for k in ("param", "grad", "m", "v", "m_e8m0", "v_e8m0"):
        assert build(entry(**{k: None}))[0] == EINVAL, k
    assert build(entry(m_e8m0=None, v_e8m0=None), bits=32)[0] == 0
    for k in ("param", "grad", "copy", "m", "v"):
        assert build(entry(**{k: 0x1008}))[0] == EALIGN, k
    assert build(entry(copy=None))[0] == 0
    assert build(entry(), short=1)[0] == EWS and build(entry(), misalign=4)[0] == EALIGN


def test_adamw_step_refusals(lib):
    def f(table=FAKE, chunks=1, bits=8, lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, step=1, lrd=None, sd=None, gd=None):
        return lib.adamw_step(table, chunks, bits, lr, b1, b2, eps, step, lrd, sd, gd, 0, 0, None)
    assert f(bits=4) == EINVAL and f(b1=1.0) == EINVAL and f(b2=-0.1) == EINVAL and f(eps=-1e-9) == EINVAL
    assert f(lr=float("inf")) == EINVAL and f(step=0) == EINVAL and f(b1=float("nan")) == EINVAL
    assert f(chunks=-1) == ESHAPE and f(chunks=1 << 24) == ESHAPE and f(table=None) == EINVAL
    assert f(table=C.c_void_p(0x1004)) == EALIGN and f(lrd=C.c_void_p(0x1002)) == EALIGN
    assert f(sd=C.c_void_p(0x1004)) == EALIGN and f(gd=C.c_void_p(0x1001)) == EALIGN
    assert f(chunks=0, table=None) == 0


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_on_the_host():
    g = torch.ones(64)
    cases = [
        (lambda: P.rmsnorm_residual_fwd(torch.zeros(4, 64), g), "x must be bf16"),
        (lambda: P.rmsnorm_residual_fwd(bf(4, 64), bf(64)), "gamma"),
        (lambda: P.rmsnorm_residual_fwd(bf(4, 64), g, want_y=False), "want_y"),
        (lambda: P.rmsnorm_residual_fwd(bf(4, 40), torch.ones(40), want_mxfp8=True), "multiple of 32"),
        (lambda: P.rmsnorm_residual_fwd(bf(4, 64), g, residual=bf(4, 32)), "residual"),
        (lambda: P.rmsnorm_residual_fwd(bf(4, 64), g, residual=torch.zeros(4, 64, dtype=torch.float16)), "residual"),
        (lambda: P.rmsnorm_residual_fwd(bf(4, 64), g, residual=bf(4, 64), z_out=torch.zeros(4, 64)), "z_out"),
        (lambda: P.rmsnorm_residual_fwd(bf(4, 64), g, z_out=bf(4, 64)), "z_out"),
        (lambda: P.rmsnorm_residual_fwd(bf(4, 64), g), "on the GPU"),
        (lambda: P.rmsnorm_residual_bwd(bf(4, 64), bf(4, 32), torch.ones(32), torch.ones(4)), "dy"),
        (lambda: P.rmsnorm_residual_bwd(bf(4, 64), bf(4, 64), g, torch.ones(5)), "rstd"),
        (lambda: P.rmsnorm_residual_bwd(bf(4, 64), bf(4, 64), g, torch.ones(4), dres=torch.zeros(4, 64)), "dres"),
        (lambda: P.swiglu_ffn_fwd(bf(4, 64), bf(64, 64), bf(64, 40)), "w13"),
        (lambda: P.swiglu_ffn_fwd(bf(4, 64), bf(64, 64), bf(32, 32)), "w2"),
        (lambda: P.swiglu_ffn_fwd(bf(4, 64), bf(64, 64), bf(64, 32), add=torch.zeros(4, 64)), "add"),
        (lambda: P.swiglu_ffn_fwd(bf(4, 64), bf(64, 64), bf(64, 32), out=bf(5, 64)), "out"),
        (lambda: P.swiglu_ffn_bwd(bf(4, 64), bf(3, 64), bf(64, 64), bf(64, 32), bf(4, 64)), "x must"),
        (lambda: P.swiglu_ffn_bwd(bf(4, 64), bf(4, 64), bf(64, 64), bf(64, 32), bf(4, 32)), "h13"),
        (lambda: P.swiglu_ffn_bwd(bf(4, 64), bf(4, 64), bf(64, 64), bf(64, 32), bf(4, 64), dw_dtype=torch.float16), "dw_dtype"),
        (lambda: P.swiglu_ffn_bwd(bf(4, 64), bf(4, 64), bf(64, 64), bf(64, 32), bf(4, 64), flags=P.BWD_DGRAD,
                                  dw13=bf(64, 64)), "BWD_WGRAD"),
        (lambda: P.swiglu_ffn_bwd(bf(4, 64), bf(4, 64), bf(64, 64), bf(64, 32), bf(4, 64), dw13=bf(64, 64)), "dw13"),
        (lambda: P.AdamWPlan([]), "at least one"),
        (lambda: P.AdamWPlan([P.AdamWTensor(bf(8), bf(8), torch.zeros(8), torch.zeros(8))]), "param"),
        (lambda: P.AdamWPlan([P.AdamWTensor(torch.zeros(8), bf(9), torch.zeros(8), torch.zeros(8))]), "grad"),
        (lambda: P.AdamWPlan([P.AdamWTensor.new(torch.zeros(8), bf(8), 8), P.AdamWTensor.new(torch.zeros(8), bf(8), 32)]),
         r"tensors\[1\].m"),
        (lambda: P.AdamWTensor.new(torch.zeros(8), bf(8), 16), "state_bits"),
    ]
    for call, what in cases:
        with pytest.raises(P.PmnError, match=what):
            call()


def test_adamw_plan_refuses_overlapping_buffers():
    """A tensor given twice, two buffers that are one, a view that reaches into another tensor's buffer
    and a gradient inside a written buffer; gradients may be shared."""
    z = torch.zeros
    p, m, g = z(64), z(64), z(64)
    one = P.AdamWTensor(p, g, m, z(64))
    for bad in ([one, one], [P.AdamWTensor(p, g, m, m)], [one, P.AdamWTensor(p[32:], z(32), z(32), z(32))],
                [P.AdamWTensor(p, p, m, z(64))]):
        with pytest.raises(P.PmnError, match="overlaps"):
            P.AdamWPlan(bad)
    with pytest.raises(P.PmnError, match="on the GPU"):   # nothing left to refuse but the CPU
        P.AdamWPlan([one, P.AdamWTensor(z(64), g, z(64), z(64))])
