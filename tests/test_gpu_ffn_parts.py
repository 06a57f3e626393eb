"""The feed-forward block for few tokens, whose products split the contraction: parts that load by pairs of stages (16
stages of 32 k or more, an even number) and by single ones (shorter, or begun inside a line), against fp64.
Bounds as derived for the other sizes of the block."""
import pytest
import torch

from test_gpu_ffn import B, U, bwd_case, case, dev, ref_bwd, ref_fwd, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import precision_moe_numerics_amd as P
    return P


# stages a part of the forward's two products, and of the backward's dy w2 and dx
SHAPES = [(100, 4088, 1024),     # 16 and 8; 8 and 16
          (40, 2048, 4096),      # 16 and 8; 8 and 16
          (33, 4096, 1400),      # 11.6 and 8.8; 8 and 11
          (300, 4096, 1024),     # 42.7 and, as 128 x 128 tiles, 16; 21.3 and, as such, 32
          (128, 2040, 2600),     # 21.3 and 10.2; 10.7 and 20.4
          (20, 1000, 2600),      # 8 and 8.2; 8 and 8.2
          (64, 512, 64)]         # 8 and 2; 8 and 4


@pytest.mark.parametrize("M,H,F", SHAPES)
def test_forward(P, M, H, F):
    d = dev(case(M, H, F, M + H + F))
    h, hb, y, yb = ref_fwd(d)
    got, h13 = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"], add=d["add"], save_h13=True)
    within(h13, h, hb, "h13")
    within(got, y, yb, "y")


@pytest.mark.parametrize("M,H,F", SHAPES)
def test_data_gradient(P, M, H, F):
    d = dev(bwd_case(M, H, F, M + H + F))
    r, e = ref_bwd(d)["dx"]
    dx = P.swiglu_ffn_bwd(d["dy"], d["x"], d["w13"], d["w2"], d["h13"], flags=P.BWD_DGRAD)[0]
    within(dx, r, e + (B + U) * (r.abs() + e), "dx")


@pytest.mark.parametrize("M,H,F", [(100, 4088, 1024), (33, 4096, 1400)])
def test_rows_keep_to_themselves(P, M, H, F):
    """A token of infinities or NaN reaches its own row: parts end inside their neighbours' k."""
    d = dev(case(M, H, F, 3, add=False))
    a = P.swiglu_ffn_fwd(d["x"], d["w13"], d["w2"])[0]
    keep = torch.arange(M, device=a.device) != 20
    for value in (float("nan"), float("inf")):
        x = d["x"].clone()
        x[20] = value
        b = P.swiglu_ffn_fwd(x, d["w13"], d["w2"])[0]
        assert torch.equal(a[keep], b[keep]) and not torch.isfinite(b[20]).any()
