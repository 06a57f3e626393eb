"""The feed-forward block on the tiles and splits that its rules choose at sizes between those of few and
of many tokens, against fp64. Bounds as derived for the other sizes of the block: K terms in fp32 are off
by (K + 2) u of their magnitudes' sum, values rounded to bf16 between the products by b = 2^-8 of
themselves, the activation's functions by 16 u (1 + |h1|).
"""
import pytest
import torch

from test_gpu_ffn import B, U, bwd_case, case, dev, ref_bwd, ref_fwd, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


# w2's product as 128 x 128 tiles in two parts, ragged at every edge
@pytest.mark.parametrize("M,H,F", [(1001, 1096, 1040), (1288, 1032, 1032)])
def test_forward_of_split_128_tiles(P, M, H, F):
    d = dev(case(M, H, F, M + H + F))
    h, hb, y, yb = ref_fwd(d)
    got, h13 = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], add=d["add"], save_h13=True)
    within(h13, h, hb, "h13")
    within(got, y, yb, "y")


# 1001, 1288: dy w2 and dx as 128 x 128 tiles in two and three parts. Few tokens: weight gradients as
# launches of 256 x 256 tiles of their own; 2056 features leave 33 of dw13's tiles to a last round in
# halves, 8456 x 2056 leaves 66 of dw13's and 50 of dw2's
@pytest.mark.parametrize("M,H,F", [(1001, 1096, 1040), (1288, 1032, 1032), (9, 4104, 1032), (9, 4104, 2056), (1, 4360, 2056),
                                   (45, 8456, 2056)])
def test_backward_of_split_128_and_lone_256_tiles(P, M, H, F):
    d = dev(bwd_case(M, H, F, M + H + F))
    ref = ref_bwd(d)
    args = (d["dy"], d["x"], d["w13"], d["w2"], d["h13"])
    for dt, half in ((torch.float32, 0.0), (torch.bfloat16, B)):
        got = dict(zip(("dx", "dw13", "dw2"), P.swiglu_ffn_bwd(*args, dw_dtype=dt)))
        for k, (r, e) in ref.items():
            within(got[k], r, e + ((B if k == "dx" else half) + U) * (r.abs() + e), f"{k} {dt}")
    for flags, keys in ((P.BWD_DGRAD, ("dx",)), (P.BWD_WGRAD, ("dw13", "dw2"))):
        one = dict(zip(("dx", "dw13", "dw2"), P.swiglu_ffn_bwd(*args, flags=flags, dw_dtype=torch.bfloat16)))
        for k in keys:
            r, e = ref[k]
            within(one[k], r, e + (B + U) * (r.abs() + e), k)
