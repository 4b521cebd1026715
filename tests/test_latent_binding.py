"""Refusals of the latent-attention binding that need no GPU: stand-ins for CUDA
tensors carry the attributes that are looked at before anything else."""
from types import SimpleNamespace

import pytest
import torch

from kimi_delta_attention_05_gb300 import latent as M


def _at(index):
    return SimpleNamespace(is_cuda=True, device=torch.device("cuda", index))


@pytest.mark.parametrize("call", [
    lambda t, s: M.latent_plan(t, t, t, t, 8, 1, stream=s), lambda t, s: M.latent_append(t, t, t, t, stream=s),
    lambda t, s: M.latent_decode(t, t, t, t, 1.0, stream=s), lambda t, s: M.latent_prefill(t, t, t, t, 1.0, stream=s),
])
def test_tensors_and_streams_of_another_device_are_refused(call, monkeypatch):
    """The library works on the current device: pointers of another one would be used on the wrong GPU."""
    monkeypatch.setattr(M, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1.*current device is cuda:0"):
        call(_at(1), None)
    with pytest.raises(ValueError, match="stream.*cuda:0.*cuda:1"):
        call(_at(0), SimpleNamespace(device=torch.device("cuda", 1)))
    monkeypatch.setattr(M, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
        call(_at(0), None)
