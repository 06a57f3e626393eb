"""Sizes of moe_grouped_gemm_bwd_bf16 that one gradient's launch holds and the other's does not, checked on the host:
only what is asked for is refused. (A pointer that is not aligned ends each call behind the check of the sizes.)"""
import ctypes as C

import precision_moe_numerics_amd as P

FAKE, ODD = C.c_void_p(0x1000), C.c_void_p(0x1008)
ESHAPE, EALIGN = -2, -3


def call(flags, G, M, N, K):
    return P._lib.moe_grouped_gemm_bwd_bf16(ODD, FAKE, M, None, FAKE, FAKE, G, M, N, K, flags, None, FAKE, 0, FAKE, 1, None, 0,
                                            None)


def test_data_gradients_of_more_matrices_than_a_weight_gradients_launch_holds():
    big = dict(G=1 << 20, M=8, N=1 << 20, K=1 << 20)
    assert call(P.BWD_WGRAD, **big) == ESHAPE and call(P.BWD_DGRAD | P.BWD_WGRAD, **big) == ESHAPE
    assert call(P.BWD_DGRAD, **big) == EALIGN


def test_weight_gradients_of_more_slots_than_a_data_gradients_launch_holds():
    big = dict(G=1, M=(1 << 31) - 8, N=8, K=1 << 20)
    assert call(P.BWD_DGRAD, **big) == ESHAPE and call(P.BWD_DGRAD | P.BWD_WGRAD, **big) == ESHAPE
    assert call(P.BWD_WGRAD, **big) == EALIGN
