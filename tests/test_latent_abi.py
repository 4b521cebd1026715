"""The latent-attention entry points refuse each invalid argument set with its
code before anything is launched (no call here has a valid one), and size their
workspaces.  Needs no GPU."""
import ctypes

import pytest
import torch

from kimi_delta_attention_05_gb300 import latent as M

FAKE = 0x7F0000000000  # 256-byte aligned, never dereferenced


def _cache(**over):
    c = M.kda_latent_cache(FAKE, 10, 64, 64 * 576, 576)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def _call(name, a, ws=None):
    fn = getattr(M._library(), f"kda_latent_{name}")
    return fn(ctypes.byref(a), None) if ws is None else fn(ctypes.byref(a), ws[0], ws[1], None)


def _set(a, over):
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    (dict(cached_lens=None), 1), (dict(slot_map=None), 1), (dict(cu_seqlens=None), 1), (dict(block_table=None), 1),
    (dict(B=-1), 3), (dict(B=16385), 3), (dict(T=-1), 3), (dict(T=1 << 31), 3), (dict(table_stride=5), 3),
    (dict(page_size=0), 17), (dict(page_size=12), 17), (dict(cu_seqlens=FAKE + 4), 9), (dict(free_pages=FAKE + 2), 9),
])
def test_plan_refusals(over, code):
    a = M.kda_latent_plan_args(FAKE, FAKE, FAKE, 6, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 6, 8, 64, 100)
    assert _call("plan", _set(a, over)) == code


@pytest.mark.parametrize("over,code", [
    (dict(c=None), 1), (dict(slot_map=None), 1), (dict(T=-1), 3), (dict(c=FAKE + 8), 9), (dict(slot_map=FAKE + 4), 9),
    (dict(c_stride=504), 15), (dict(c_stride=580), 15), (dict(k_pe_stride=60), 15),
    (dict(cache=_cache(page_size=20)), 17), (dict(cache=_cache(data=None)), 1), (dict(cache=_cache(data=FAKE + 8)), 9),
    (dict(cache=_cache(token_stride=572)), 15), (dict(cache=_cache(page_stride=63 * 576)), 15),
    (dict(cache=_cache(num_pages=-1)), 3),
])
def test_append_refusals(over, code):
    a = M.kda_latent_append_args(FAKE, FAKE, 576, 576, FAKE, _cache(), None, 1e-6, 7)
    assert _call("append", _set(a, over)) == code


def test_append_of_no_tokens_is_nothing():
    assert _call("append", M.kda_latent_append_args(None, None, 0, 0, None, _cache(), None, 1e-6, 0)) == 0


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(seq_lens=None), 1), (dict(block_table=None), 1),
    (dict(B=-1), 3), (dict(R=5000), 3), (dict(H=1 << 20), 3), (dict(table_stride=3), 3), (dict(max_pages=1 << 30), 3),
    (dict(scale=0.0), 16), (dict(scale=-1.0), 16), (dict(scale=float("nan")), 16), (dict(scale=float("inf")), 16),
    (dict(q=FAKE + 8), 9), (dict(out=FAKE + 2), 9), (dict(seq_lens=FAKE + 2), 9), (dict(lse=FAKE + 2), 9),
    (dict(cache=_cache(page_size=100)), 17), (dict(cache=_cache(token_stride=570)), 15),
])
def test_decode_refusals(over, code):
    a = M.kda_latent_decode_args(FAKE, _cache(), FAKE, 4, 4, FAKE, 0.07, FAKE, None, 2, 1, 32)
    a = _set(a, over)
    a.table_stride = max(a.table_stride, a.max_pages) if "max_pages" in over else a.table_stride
    assert _call("decode", a, (FAKE, 1 << 40)) == code
    assert M._library().kda_latent_decode_workspace_bytes(ctypes.byref(a)) == 0


def test_decode_workspace_is_checked():
    a = M.kda_latent_decode_args(FAKE, _cache(), FAKE, 4, 4, FAKE, 0.07, FAKE, None, 2, 1, 32)
    need = M._library().kda_latent_decode_workspace_bytes(ctypes.byref(a))
    if need:
        assert _call("decode", a, (None, need)) == 10
        assert _call("decode", a, (FAKE, need - 1)) == 10
        assert _call("decode", a, (FAKE + 16, need)) == 10


def test_decode_workspace_of_long_tables_is_checked():
    """Tables that one CTA does not walk alone hold parts to be joined."""
    a = M.kda_latent_decode_args(FAKE, _cache(), FAKE, 400, 400, FAKE, 0.07, FAKE, None, 2, 1, 32)
    need = M._library().kda_latent_decode_workspace_bytes(ctypes.byref(a))
    assert need > 0
    assert _call("decode", a, (None, need)) == 10
    assert _call("decode", a, (FAKE, need - 1)) == 10
    assert _call("decode", a, (FAKE + 16, need)) == 10


def test_decode_of_nothing_is_nothing():
    a = M.kda_latent_decode_args(None, _cache(), None, 0, 0, None, 0.07, None, None, 0, 1, 32)
    assert _call("decode", a, (None, 0)) == 0


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(v=None), 1), (dict(k_pe=None), 1), (dict(cu_seqlens_k=None), 1),
    (dict(B=2), 8), (dict(Tq=-1), 3), (dict(H=70000), 3), (dict(Tk=1 << 31), 3), (dict(flags=2), 4),
    (dict(scale=0.0), 16), (dict(scale=float("nan")), 16), (dict(q=FAKE + 8), 9), (dict(cu_seqlens_q=FAKE + 4), 9),
    (dict(q_stride_h=184), 15), (dict(k_stride_t=100), 15), (dict(v_stride_h=129), 15), (dict(k_pe_stride_t=32), 15),
])
def test_prefill_refusals(over, code):
    a = M.kda_latent_prefill_args(FAKE, FAKE, FAKE, FAKE, 768, 192, 1024, 256, 64, 1024, 256, 0.07, FAKE, None, FAKE, FAKE,
                                  1, 100, 120, 4, 3, 1)
    assert _call("prefill", _set(a, over), (FAKE, 1 << 40)) == code


def test_prefill_dense_batch_and_workspace():
    a = M.kda_latent_prefill_args(FAKE, FAKE, FAKE, FAKE, 768, 192, 1024, 256, 64, 1024, 256, 0.07, FAKE, None, None, None,
                                  2, 100, 120, 4, 3, 1)
    assert _call("prefill", a, (FAKE, 1 << 40)) == 3  # N != B
    a.cu_seqlens_q = a.cu_seqlens_k = FAKE
    a.B = 1
    need = M._library().kda_latent_prefill_workspace_bytes(ctypes.byref(a))
    assert need > 0 and _call("prefill", a, (FAKE, need - 1)) == 10 and _call("prefill", a, (FAKE + 16, need)) == 10


def test_tensors_that_are_not_on_a_gpu_are_refused():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        M.latent_plan(z(1, dtype=torch.int32), z(1, dtype=torch.int32), z(1, 1, dtype=torch.int32), z(1, dtype=torch.int32), 8, 1)
    with pytest.raises(ValueError, match="CUDA"):
        M.latent_append(z(1, 512), z(1, 64), z(1, dtype=torch.int64), z(1, 8, 576))
    with pytest.raises(ValueError, match="CUDA"):
        M.latent_decode(z(1, 1, 1, 576), z(1, 8, 576), z(1, 1, dtype=torch.int32), z(1, dtype=torch.int32), 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        M.latent_prefill(z(1, 1, 1, 192), z(1, 1, 1, 128), z(1, 1, 64), z(1, 1, 1, 128), 1.0)
