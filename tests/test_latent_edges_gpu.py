"""Latent attention on the GPU at the edges of what its interface accepts:
buffers at the smallest alignment, and the forms that large calls take."""
import numpy as np
import pytest
import torch

from kimi_delta_attention_05_gb300 import KdaError, get_status, latent as M
from tests.test_latent_gpu import NAN, _rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    get_status()
    yield


# ---- prefill: an `out` on a 16-byte boundary that is not one of 32 ----

@pytest.mark.parametrize("lq,lk,heads,packed", [
    ([300], [300], 3, False),                       # single CTAs
    ([1100], [1100], 2, False),                     # pairs
    ([130, 1, 300], [130, 7, 310], 2, True),        # packed, single CTAs
    ([2300, 1900], [2300, 1900], 1, True),          # packed, pairs
    ([300], [4200], 100, False),                    # split over the keys, single CTAs: whole items and parts
    ([1100], [4300], 32, False),                    # split, pairs
    ([1, 130, 300], [5000, 4300, 9000], 2, True),   # packed and split
    ([2100], [9000], 1, True),                      # packed and split, pairs
])
@pytest.mark.parametrize("at", [8, 24])
def test_prefill_writes_an_out_of_any_16_bytes(lq, lk, heads, packed, at):
    """The same bits as into a buffer of the allocator's, and nothing beside it."""
    gen = torch.Generator().manual_seed(sum(lq) + at)
    if not packed:
        assert (M.latent_prefill_workspace_bytes(1, lq[0], lk[0], heads) > 0) == (lk[0] > 4096)
    q, k, pe, v = (_rand(gen, 1, *x).cuda() for x in ((sum(lq), heads, 192), (sum(lk), heads, 128), (sum(lk), 64),
                                                      (sum(lk), heads, 128)))
    cu = [torch.tensor([0] + list(np.cumsum(x)), device="cuda") for x in (lq, lk)] if packed else [None, None]
    lse, again = (torch.full((1, sum(lq), heads), NAN, device="cuda") for _ in range(2))
    ref = M.latent_prefill(q, k, pe, v, 0.07, lse=lse, cu_seqlens=cu[0], cu_seqlens_k=cu[1])
    n = ref.numel()
    buf = torch.full((n + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[at:at + n].view(ref.shape)
    assert ref.data_ptr() % 32 == 0 and out.data_ptr() % 32 == 16
    assert M.latent_prefill(q, k, pe, v, 0.07, out=out, lse=again, cu_seqlens=cu[0], cu_seqlens_k=cu[1]) is out
    assert torch.equal(out, ref) and torch.equal(again, lse)
    assert (buf[:at] == 5.0).all() and (buf[at + n:] == 5.0).all()
    assert get_status() == 0


# ---- refusals of the binding ----

def test_workspaces_that_the_gpu_cannot_write_are_refused():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    decode = z(2, 1, 4, 576), z(80, 8, 576), z(2, 40, d=torch.int32), z(2, d=torch.int32)
    prefill = z(1, 5, 3, 192), z(1, 5, 3, 128), z(1, 5, 64), z(1, 5, 3, 128)
    cu = torch.tensor([0, 5], device="cuda")
    for ws in (torch.empty(1 << 24, dtype=torch.uint8), z(1, d=torch.uint8).expand(1 << 24), z(1 << 24, d=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            M.latent_decode(*decode, 1.0, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            M.latent_prefill(*prefill, 1.0, cu_seqlens=cu, workspace=ws)
    ws = z(1 << 22, d=torch.float32)
    assert torch.equal(M.latent_decode(*decode, 1.0, workspace=ws), M.latent_decode(*decode, 1.0))


@pytest.mark.parametrize("scale", [1e39, float("inf"), float("nan"), -1e39, 0, 1e-60])
def test_scales_that_are_not_positive_32_bit_numbers_are_refused(scale):
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    with pytest.raises(KdaError, match="kda_latent_decode.*16"):
        M.latent_decode(z(2, 1, 4, 576), z(8, 8, 576), z(2, 4, d=torch.int32), z(2, d=torch.int32), scale)
    with pytest.raises(KdaError, match="kda_latent_prefill.*16"):
        M.latent_prefill(z(1, 5, 3, 192), z(1, 5, 3, 128), z(1, 5, 64), z(1, 5, 3, 128), scale)
