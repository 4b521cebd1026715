"""Refusals of the latent-attention calls that need no GPU: stand-ins for CUDA tensors
carry the attributes that the binding looks at before anything else; the library
is called with addresses that it never follows."""
import ctypes
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


FAKE = 0x7F0000000000


@pytest.mark.parametrize("tq,tk,code", [(100, 120, 14), (0, 120, 14), (100, 0, 14), (0, 0, 0)])
def test_packed_tokens_without_sequences_are_refused(tq, tk, code):
    """Offsets of one entry cannot be 0 and T: `out` would be returned as it was allocated."""
    a = M.kda_latent_prefill_args(FAKE, FAKE, FAKE, FAKE, 768, 192, 1024, 256, 64, 1024, 256, 0.07, FAKE, None, FAKE, FAKE,
                                  1, tq, tk, 4, 0, 1)
    lib = M._library()
    assert lib.kda_latent_prefill(ctypes.byref(a), FAKE, 1 << 40, None) == code
    assert lib.kda_latent_prefill_workspace_bytes(ctypes.byref(a)) == (0 if code else 256)


def test_more_packed_blocks_than_32_bits_count_are_refused():
    """Before anything is launched, as every argument error; empty sequences make it possible for small tensors."""
    a = M.kda_latent_prefill_args(FAKE, FAKE, FAKE, FAKE, 192 * 1024, 192, 256 * 1024, 256, 64, 256 * 1024, 256, 0.07, FAKE,
                                  None, FAKE, FAKE, 1, 100, 100, 1024, 1 << 22, 1)
    lib = M._library()
    assert lib.kda_latent_prefill(ctypes.byref(a), FAKE, 1 << 40, None) == 3
    a.H = 500
    assert lib.kda_latent_prefill_workspace_bytes(ctypes.byref(a)) > 0


def test_workspaces_that_the_gpu_cannot_write_are_refused():
    """Not on the device, or more elements than memory (an expanded view)."""
    cpu = torch.device("cpu")
    assert M._scratch(None, cpu) == (None, 0)
    ws = torch.empty(512, dtype=torch.uint8)
    assert M._scratch(ws, cpu) == (ws.data_ptr(), 512)
    assert M._scratch(torch.empty(8, dtype=torch.float32), cpu)[1] == 32
    with pytest.raises(ValueError, match="workspace"):
        M._scratch(ws, torch.device("cuda", 0))
    for view in (ws[:1].expand(1 << 20), ws[::2]):
        with pytest.raises(ValueError, match="workspace"):
            M._scratch(view, cpu)


def test_the_binding_asks_for_a_workspace_from_the_keys_on_from_which_calls_are_split():
    """The limit stands in the header and in the binding: were the binding's higher, calls between the two
    would silently run whole."""
    for rows, heads in ((1, 1), (200, 1)):
        assert M.latent_prefill_workspace_bytes(1, rows, M._SPLIT_KEYS - 1, heads) == 0
        assert M.latent_prefill_workspace_bytes(1, rows, M._SPLIT_KEYS, heads) > 0
