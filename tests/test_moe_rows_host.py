"""Refusals of the expert layer's operators on unquantized activations, checked on the host before anything is
launched: through the C ABI with pointers that are never dereferenced, and through the binding with tensors on
the CPU."""
import ctypes as C

import pytest
import torch

import precision_moe_numerics_amd as P

FAKE, ODD = C.c_void_p(0x1000), C.c_void_p(0x1008)
EINVAL, ESHAPE, EALIGN, EWS = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    return P._lib


def test_grouped_forward_refusals(lib):
    def f(x=FAKE, rows=8, gather=None, w=FAKE, off=FAKE, G=2, M=8, N=64, K=64, epi=1, out=FAKE, aux=None):
        return lib.moe_grouped_gemm_fwd_bf16(x, rows, gather, w, off, G, M, N, K, epi, out, aux, None)
    assert f(epi=3) == EINVAL and f(epi=-1) == EINVAL
    assert f(G=0) == ESHAPE and f(M=-1) == ESHAPE and f(M=1 << 31, rows=1 << 31) == ESHAPE and f(rows=7) == ESHAPE
    assert f(rows=-1, gather=FAKE) == ESHAPE and f(N=60) == ESHAPE and f(K=68) == ESHAPE and f(N=0) == ESHAPE and f(K=0) == ESHAPE
    assert f(N=72, epi=2) == ESHAPE and f(N=(1 << 20) + 8) == ESHAPE and f(K=(1 << 20) + 8) == ESHAPE
    assert f(M=1 << 30, rows=1 << 30, N=1 << 20) == ESHAPE       # a launch holds fewer than 2^32 threads
    for k in ("x", "w", "off", "out"):
        assert f(**{k: None}) == EINVAL, k
    for k in ("x", "w", "out", "aux"):
        assert f(**{k: ODD}) == EALIGN, k
    assert f(gather=C.c_void_p(0x1002)) == EALIGN and f(off=C.c_void_p(0x1004)) == EALIGN
    assert f(M=0, rows=0, x=None, out=None, off=None) == 0


def test_grouped_backward_refusals(lib):
    size = lib.moe_grouped_gemm_bwd_bf16_workspace_size
    assert size(8, 2, 64, 64, 3, 0) == 0 and size(8, 2, 64, 64, 1, 1) == 0 and size(0, 2, 64, 64, 3, 1) == 0
    assert size(8, 2, 64, 64, 2, 1) >= 8 * 64 * 2 and size(-1, 2, 64, 64, 3, 1) == 0 and size(8, 0, 64, 64, 3, 1) == 0
    n = size(8, 2, 64, 64, 3, 1)
    # few and small matrices over many slots: the parts' sums, at least two
    few = size(4096, 2, 64, 64, 2, 0)
    assert few >= 2 * 2 * 64 * 64 * 4 and size(4096, 2, 64, 64, 2, 1) == few + 4096 * 64 * 2
    assert size(4096, 2, 64, 64, 1, 0) == 0 and size(65536, 48, 4096, 4096, 3, 0) == 0

    def f(dy=FAKE, x=FAKE, rows=8, gather=None, w=FAKE, off=FAKE, G=2, M=8, N=64, K=64, flags=3, h13=None, da=FAKE, dat=0,
          db=FAKE, dbt=1, ws=None, nb=0):
        return lib.moe_grouped_gemm_bwd_bf16(dy, x, rows, gather, w, off, G, M, N, K, flags, h13, da, dat, db, dbt, ws, nb, None)
    assert f(flags=0) == EINVAL and f(flags=4) == EINVAL and f(flags=3 | 8) == EINVAL
    assert f(dat=2) == EINVAL and f(dbt=-1) == EINVAL and f(h13=FAKE, dat=1) == EINVAL
    assert f(h13=FAKE, gather=FAKE) == EINVAL and f(h13=FAKE, flags=2) == EINVAL
    assert f(G=0) == ESHAPE and f(M=-1) == ESHAPE and f(N=4) == ESHAPE and f(K=20) == ESHAPE and f(rows=7) == ESHAPE
    assert f(G=1 << 20, N=1 << 20, K=1 << 20) == ESHAPE
    for k in ("dy", "x", "w", "off", "da", "db"):
        assert f(**{k: None}) == EINVAL, k
    assert f(x=None, h13=FAKE) == EWS and f(x=None, h13=FAKE, ws=FAKE, nb=n - 1) == EWS
    assert f(M=4096, rows=4096) == EWS and f(M=4096, rows=4096, ws=FAKE, nb=few - 1) == EWS
    assert f(M=4096, rows=4096, ws=ODD, nb=few) == EALIGN
    for k in ("dy", "x", "w", "h13", "da", "db"):
        assert f(**{k: ODD}) == EALIGN, k
    assert f(x=None, h13=FAKE, ws=ODD, nb=n) == EALIGN and f(gather=C.c_void_p(0x1002)) == EALIGN
    assert f(M=0, rows=0, flags=1, dy=None, x=None) == 0


def test_gemv_refusals(lib):
    size = lib.moe_gemv_nvfp4_workspace_size
    assert size(17, 2, 64, 0) == 0 and size(0, 2, 64, 1) == 0 and size(17, 2, 64, 1) >= 17 * 2 * 64 * 4

    def f(x=FAKE, pp=0, c=FAKE, s=FAKE, o=FAKE, rpo=64, ids=FAKE, gates=None, add=None, T=4, k=2, G=8, N=64, K=64, epi=1,
          out=FAKE, ws=None, nb=0):
        return lib.moe_gemv_nvfp4(x, pp, c, s, o, rpo, ids, gates, add, T, k, G, N, K, epi, out, ws, nb, None)
    assert f(epi=3) == EINVAL and f(gates=FAKE, epi=2) == EINVAL and f(add=FAKE) == EINVAL
    assert f(ids=None) == EINVAL and f(ids=None, G=1) == EINVAL and f(ids=None, k=1) == EINVAL
    assert f(T=-1) == ESHAPE and f(k=0) == ESHAPE and f(G=0) == ESHAPE and f(N=48) == ESHAPE and f(K=48) == ESHAPE
    assert f(N=96, epi=2) == ESHAPE and f(rpo=16) == ESHAPE and f(rpo=0) == ESHAPE and f(rpo=40) == ESHAPE
    assert f(T=4097, k=1) == ESHAPE and f(T=2049, k=2) == ESHAPE and f(T=1 << 40) == ESHAPE and f(N=0) == ESHAPE
    assert f(T=4096, k=1, G=4096, N=1 << 20) == ESHAPE and f(epi=2, N=1 << 17, K=(1 << 16) + 32) == ESHAPE
    for q in ("x", "c", "s", "o", "out"):
        assert f(**{q: None}) == EINVAL, q
    assert f(T=20, gates=FAKE) == EWS and f(T=20, gates=FAKE, ws=FAKE, nb=size(20, 2, 64, 1) - 1) == EWS
    assert f(T=20, gates=FAKE, ws=ODD, nb=size(20, 2, 64, 1)) == EALIGN
    for q in ("x", "c", "out"):
        assert f(**{q: ODD}) == EALIGN, q
    assert f(gates=FAKE, add=ODD, ws=FAKE, nb=size(4, 2, 64, 1)) == EALIGN and f(s=ODD) == EALIGN and f(ids=C.c_void_p(0x1002)) == EALIGN
    assert f(T=0, x=None, out=None) == 0


def test_combine_refusals(lib):
    def f(y=FAKE, yt=0, M=8, H=64, so=FAKE, g=FAKE, add=None, T=4, k=2, out=FAKE, ot=0):
        return lib.moe_combine_rows_fwd(y, yt, M, H, so, g, add, T, k, out, ot, None)

    def b(d=FAKE, dt=0, y=FAKE, yt=0, M=8, H=64, so=FAKE, g=FAKE, T=4, k=2, dy=FAKE, dg=FAKE):
        return lib.moe_combine_rows_bwd(d, dt, y, yt, M, H, so, g, T, k, dy, dg, None)
    assert f(yt=2) == EINVAL and f(ot=-1) == EINVAL and b(dt=2) == EINVAL and b(yt=3) == EINVAL
    for q in (f, b):
        assert q(M=-1) == ESHAPE and q(M=1 << 31) == ESHAPE and q(H=60) == ESHAPE and q(H=-8) == ESHAPE
        assert q(H=(1 << 20) + 8) == ESHAPE and q(T=-1) == ESHAPE and q(T=1 << 24) == ESHAPE
        assert q(k=0) == ESHAPE and q(k=65) == ESHAPE and q(so=None, M=7) == ESHAPE
        assert q(y=None) == EINVAL and q(y=ODD) == EALIGN and q(so=C.c_void_p(0x1002)) == EALIGN and q(g=C.c_void_p(0x1001)) == EALIGN
    assert f(out=None) == EINVAL and f(out=ODD) == EALIGN and f(add=ODD) == EALIGN
    assert b(dy=None, dg=None) == EINVAL and b(d=None) == EINVAL and b(d=ODD) == EALIGN and b(dy=ODD) == EALIGN
    assert b(dg=C.c_void_p(0x1002)) == EALIGN
    assert f(T=0, y=None, out=None) == 0 and b(T=0, d=None, y=None) == 0


def test_combine_backward_of_nothing(lib):
    """Tensors without values have no address: no tokens, or no rows and no dgates, is no error."""
    f = lambda T, M, dy, dg: lib.moe_combine_rows_bwd(FAKE, 0, FAKE, 0, M, 64, FAKE, FAKE, T, 2, dy, dg, None)  # noqa: E731
    assert f(0, 0, None, None) == 0 and f(0, 8, FAKE, None) == 0 and f(4, 0, None, None) == 0
    assert f(4, 8, None, None) == EINVAL


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_on_the_host():
    off = torch.tensor([0, 3, 8])
    f32 = torch.zeros
    w = bf(2 * 64, 32)
    for bad in (lambda: P.moe_grouped_gemm_fwd_bf16(f32(8, 32), w, off, 8, 64),
                lambda: P.moe_grouped_gemm_fwd_bf16(bf(8, 40), w, off, 8, 64),
                lambda: P.moe_grouped_gemm_fwd_bf16(bf(8, 32), bf(64, 32), off, 8, 64),
                lambda: P.moe_grouped_gemm_fwd_bf16(bf(8, 32), w, off.int(), 8, 64),
                lambda: P.moe_grouped_gemm_fwd_bf16(bf(8, 32), w, off, 8, 64, P.EPI_RHT32_S2F6),
                lambda: P.moe_grouped_gemm_fwd_bf16(bf(8, 32), w, off, 8, 64, gather=i32(7)),
                lambda: P.moe_grouped_gemm_bwd_bf16(bf(8, 32), bf(8, 32), w, off, 8, 64),
                lambda: P.moe_grouped_gemm_bwd_bf16(bf(8, 64), None, w, off, 8, 64),
                lambda: P.moe_grouped_gemm_bwd_bf16(bf(8, 64), bf(8, 32), w, off, 8, 64, da_dtype=torch.float16),
                lambda: P.moe_grouped_gemm_bwd_bf16(bf(8, 64), bf(8, 32), w, off, 8, 64, h13=bf(8, 32)),
                lambda: P.moe_grouped_gemm_bwd_bf16(bf(8, 64), bf(8, 32), w, off, 8, 64, h13=bf(8, 64), gather=i32(8)),
                lambda: P.moe_grouped_gemm_bwd_bf16(bf(8, 64), bf(8, 32), w, off, 8, 64, flags=P.BWD_WGRAD, da=bf(8, 32)),
                lambda: P.moe_combine_rows_fwd(bf(8, 64), i32(4, 2).long()),
                lambda: P.moe_combine_rows_fwd(bf(8, 64).half(), i32(4, 2)),
                lambda: P.moe_combine_rows_fwd(bf(8, 64), i32(4, 2), f32(4, 3)),
                lambda: P.moe_combine_rows_fwd(bf(8, 64), i32(4, 2), add=f32(4, 64)),
                lambda: P.moe_combine_rows_bwd(bf(3, 64), bf(8, 64), i32(4, 2)),
                lambda: P.moe_combine_rows_bwd(bf(4, 64), bf(8, 64), i32(4, 2), want_dy=False, want_dgates=False),
                lambda: P.moe_combine_rows_bwd(bf(4, 64), bf(8, 64), i32(4, 2), want_dy=False, dy=bf(8, 64)),
                # tensors that are not on the GPU
                lambda: P.moe_grouped_gemm_fwd_bf16(bf(8, 32), w, off, 8, 64),
                lambda: P.moe_grouped_gemm_bwd_bf16(bf(8, 64), bf(8, 32), w, off, 8, 64),
                lambda: P.moe_combine_rows_fwd(bf(8, 64), i32(4, 2)),
                lambda: P.moe_combine_rows_bwd(bf(4, 64), bf(8, 64), i32(4, 2))):
        with pytest.raises(P.PmnError):
            bad()


def test_gemv_binding_refuses_on_the_host():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    wq = P.NVFP4(u8(3 * 64, 32), u8(3 * 64, 4), torch.ones(3), 64)
    x, ids, gates = bf(4, 64), i32(4, 2), torch.zeros(4, 2)
    for kw in (dict(x=x.float()), dict(x=bf(4, 32)), dict(x=bf(4, 3, 64)), dict(N=48), dict(ids=ids.long()), dict(ids=i32(3, 2)),
               dict(ids=None), dict(epilogue=P.EPI_RHT32_S2F6), dict(gates=torch.zeros(4, 3)),
               dict(gates=gates, epilogue=P.EPI_SWIGLU), dict(add=bf(4, 64)), dict(gates=gates, add=bf(4, 32)), {}):
        a = dict(x=x, wq=wq, N=64, ids=ids)
        a.update(kw)
        with pytest.raises(P.PmnError):
            P.moe_gemv_nvfp4(**a)
