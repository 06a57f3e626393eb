"""The binding's check of a tensor's device against the current one, on the host: it asks torch's public interface."""
import pytest
import torch

import precision_moe_numerics_amd as P


class At:
    """What the check reads of a tensor."""

    def __init__(self, device):
        self.device_index = device

    def get_device(self):
        return self.device_index


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    assert P._device_of(At(2), "x") == 2
    with pytest.raises(P.PmnError, match="x is on cuda:0, the current device is cuda:2"):
        P._device_of(At(0), "x")
    with pytest.raises(P.PmnError, match="must be on the GPU"):
        P._device_of(At(-1), "x")
