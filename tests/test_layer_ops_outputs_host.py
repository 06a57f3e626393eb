"""Refusals of outputs that the caller gives to the operators around the routed experts, on the host."""
import pytest
import torch

import precision_moe_numerics_amd as P


def test_given_dgamma_is_checked():
    z, g, s = torch.zeros((4, 64), dtype=torch.bfloat16), torch.ones(64), torch.ones(4)
    for bad in (torch.zeros(63), torch.zeros(64, dtype=torch.bfloat16), torch.zeros((1, 64))):
        with pytest.raises(P.PmnError, match="dgamma"):
            P.rmsnorm_residual_bwd(z, z, g, s, dgamma=bad)
    with pytest.raises(P.PmnError, match="on the GPU"):
        P.rmsnorm_residual_bwd(z, z, g, s, dgamma=torch.zeros(64))
