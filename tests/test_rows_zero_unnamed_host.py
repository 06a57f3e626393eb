"""Refusals of moe_rows_zero_unnamed, checked on the host before anything is launched."""
import ctypes as C

import pytest
import torch

import precision_moe_numerics_amd as P

FAKE, ODD = C.c_void_p(0x1000), C.c_void_p(0x1008)
EINVAL, ESHAPE, EALIGN = -1, -2, -3


def test_refusals():
    def f(x=FAKE, xt=0, M=8, H=64, so=FAKE, T=4, k=2):
        return P._lib.moe_rows_zero_unnamed(x, xt, M, H, so, T, k, None)
    assert f(xt=2) == EINVAL and f(xt=-1) == EINVAL and f(x=None) == EINVAL and f(so=None) == EINVAL
    assert f(M=-1) == ESHAPE and f(M=1 << 31) == ESHAPE and f(H=60) == ESHAPE and f(H=(1 << 20) + 8) == ESHAPE
    assert f(T=-1) == ESHAPE and f(T=1 << 24) == ESHAPE and f(k=0) == ESHAPE and f(k=65) == ESHAPE
    assert f(x=ODD) == EALIGN and f(so=C.c_void_p(0x1002)) == EALIGN
    assert f(M=0, x=None) == 0 and f(H=0, x=None) == 0


def test_binding_refuses_on_the_host():
    x, so = torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((4, 2), dtype=torch.int32)
    for bad in (lambda: P.moe_rows_zero_unnamed(x.half(), so), lambda: P.moe_rows_zero_unnamed(x[0], so),
                lambda: P.moe_rows_zero_unnamed(x, so.long()), lambda: P.moe_rows_zero_unnamed(x, so.view(-1)),
                lambda: P.moe_rows_zero_unnamed(x, so)):      # the last: not on the GPU
        with pytest.raises(P.PmnError):
            bad()
