"""The calls on shared pages refuse each invalid argument set with its code before
anything is launched, and the binding what it can see.  Needs no GPU."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from kimi_delta_attention_05_gb300 import latent as M
from kimi_delta_attention_05_gb300 import latent_pages as G

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


BAD_CACHES = [(dict(cache=_cache(page_size=20)), 17), (dict(cache=_cache(data=None)), 1), (dict(cache=_cache(data=FAKE + 8)), 9),
              (dict(cache=_cache(token_stride=572)), 15), (dict(cache=_cache(page_stride=63 * 576)), 15),
              (dict(cache=_cache(num_pages=-1)), 3)]


@pytest.mark.parametrize("over,code", [
    (dict(parents=None), 1), (dict(children=None), 1), (dict(cached_lens=None), 1), (dict(block_table=None), 1),
    (dict(shares=None), 1), (dict(seq_lens=None), 1), (dict(pages_taken=None), 1), (dict(free_pages=None), 1),
    (dict(F=-1), 3), (dict(F=16385), 3), (dict(B=16385), 3), (dict(num_free=-1), 3), (dict(table_stride=5), 3),
    (dict(shares=FAKE + 2), 9), (dict(fork_lens=FAKE + 1), 9), (dict(block_table=FAKE + 2), 9),
] + BAD_CACHES)
def test_fork_refusals(over, code):
    a = G.kda_latent_fork_args(FAKE, FAKE, FAKE, FAKE, FAKE, 6, FAKE, FAKE, _cache(), FAKE, FAKE, 2, 4, 6, 8)
    assert _call("fork", _set(a, over)) == code


@pytest.mark.parametrize("over,code", [
    (dict(rows=None), 1), (dict(cached_lens=None), 1), (dict(block_table=None), 1), (dict(shares=None), 1),
    (dict(seq_lens=None), 1), (dict(pages=None), 1), (dict(count=None), 1), (dict(F=-1), 3), (dict(F=16385), 3),
    (dict(B=-1), 3), (dict(num_pages=1 << 31), 3), (dict(max_pages=-1), 3), (dict(table_stride=5), 3),
    (dict(page_size=0), 17), (dict(page_size=12), 17), (dict(rows=FAKE + 2), 9), (dict(pages=FAKE + 1), 9),
])
def test_release_refusals(over, code):
    a = G.kda_latent_release_args(FAKE, FAKE, FAKE, FAKE, 6, FAKE, FAKE, FAKE, FAKE, 2, 4, 6, 10, 64)
    assert _call("release", _set(a, over)) == code


def _compact_args(**over):
    return _set(G.kda_latent_compact_args(FAKE, FAKE, 6, FAKE, 6, FAKE, FAKE, FAKE, FAKE, _cache(), 4, 6), over)


@pytest.mark.parametrize("over,code", [
    (dict(cached_lens=None), 1), (dict(block_table=None), 1), (dict(block_table_out=None), 1), (dict(shares=None), 1),
    (dict(shares_out=None), 1), (dict(page_map=None), 1), (dict(pages_used=None), 1), (dict(B=-1), 3), (dict(B=16385), 3),
    (dict(table_stride=5), 3), (dict(table_out_stride=5), 3), (dict(page_map=FAKE + 2), 9),
    (dict(cache=_cache(num_pages=12582913)), 3),
] + BAD_CACHES)
def test_compact_refusals(over, code):
    assert _call("compact", _compact_args(**over)) == code


@pytest.mark.parametrize("over,code", [
    (dict(src_pages=None), 1), (dict(dst_pages=None), 1), (dict(n=-1), 3), (dict(n=1 << 31), 3),
    (dict(src_pages=FAKE + 2), 9), (dict(src=_cache(page_size=32)), 17), (dict(dst=_cache(token_stride=570)), 15),
    (dict(src=_cache(data=None)), 1),
])
def test_copy_refusals(over, code):
    a = G.kda_latent_copy_args(_cache(), _cache(), FAKE, FAKE, 3)
    assert _call("copy", _set(a, over)) == code


def test_copy_of_no_pages_is_nothing():
    assert _call("copy", G.kda_latent_copy_args(_cache(), _cache(), None, None, 0)) == 0


CALLS = {
    "fork": lambda t, s=None: G.latent_fork(t, t, t, t, t, t, t, stream=s),
    "release": lambda t, s=None: G.latent_release(t, t, t, t, 8, stream=s),
    "compact": lambda t, s=None: G.latent_compact(t, t, t, t, stream=s),
    "copy": lambda t, s=None: G.latent_copy(t, t, t, t, stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_another_place_are_refused(name, monkeypatch):
    with pytest.raises(ValueError, match="CUDA"):
        CALLS[name](torch.zeros(1, dtype=torch.int32))
    at = lambda i: SimpleNamespace(is_cuda=True, device=torch.device("cuda", i))  # noqa: E731
    monkeypatch.setattr(M, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1.*current device is cuda:0"):
        CALLS[name](at(1))
    with pytest.raises(ValueError, match="stream.*cuda:0.*cuda:1"):
        CALLS[name](at(0), SimpleNamespace(device=torch.device("cuda", 1)))


def _shared_args(over):
    d = M.kda_latent_decode_args(FAKE, _cache(), FAKE, 4, 4, FAKE, 0.07, FAKE, None, 2, 1, 32)
    a = M.kda_latent_decode_shared_args(d, FAKE, FAKE, 1)
    for k, v in over.items():
        setattr(a.decode if hasattr(d, k) else a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(seq_lens=None), 1), (dict(block_table=None), 1), (dict(cu_groups=None), 1),
    (dict(prefix_lens=None), 1), (dict(B=-1), 3), (dict(G=-1), 3), (dict(G=16385), 3), (dict(G=0), 14),
    (dict(B=1 << 20, H=4096), 3), (dict(max_pages=(1 << 24) + 1, table_stride=1 << 25), 3), (dict(table_stride=3), 3), (dict(scale=0.0), 16), (dict(cu_groups=FAKE + 4), 9),
    (dict(prefix_lens=FAKE + 2), 9), (dict(q=FAKE + 8), 9), (dict(cache=_cache(page_size=100)), 17),
    (dict(cache=_cache(token_stride=570)), 15),
])
def test_decode_shared_refusals(over, code):
    a = _shared_args(over)
    assert _call("decode_shared", a, (FAKE, 1 << 50)) == code
    assert M._library().kda_latent_decode_shared_workspace_bytes(ctypes.byref(a)) == 0


def test_decode_shared_workspace_is_checked():
    a = _shared_args(dict(max_pages=400, table_stride=400))
    need = M._library().kda_latent_decode_shared_workspace_bytes(ctypes.byref(a))
    assert need > 0
    for ws in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert _call("decode_shared", a, ws) == 10


def test_decode_shared_of_nothing_is_nothing():
    d = M.kda_latent_decode_args(None, _cache(), None, 0, 0, None, 0.07, None, None, 0, 1, 32)
    assert _call("decode_shared", M.kda_latent_decode_shared_args(d, FAKE, None, 0), (None, 0)) == 0


def test_decode_shared_refuses_tensors_of_another_place():
    with pytest.raises(ValueError, match="CUDA"):
        t = torch.zeros(1, dtype=torch.int32)
        M.latent_decode_shared(torch.zeros(1, 1, 1, 576), t, t, t, t, t, 1.0)


@pytest.mark.parametrize("max_pages", [0, 4, 40000])
@pytest.mark.parametrize("B,R,H", [(2, 0, 16), (2, 1, 0), (2000, 0, 0), (0, 1, 32), (0, 0, 0)])
def test_decode_shared_without_rows_is_nothing_whatever_the_table(B, R, H, max_pages):
    """As kda_latent_decode: no workspace, no launch."""
    d = M.kda_latent_decode_args(FAKE, _cache(), FAKE, max_pages, max_pages, FAKE, 0.07, FAKE, None, B, R, H)
    a = M.kda_latent_decode_shared_args(d, FAKE, FAKE, 1)
    assert M._library().kda_latent_decode_shared_workspace_bytes(ctypes.byref(a)) == 0
    assert _call("decode", d, (None, 0)) == 0 and _call("decode_shared", a, (None, 0)) == 0


@pytest.mark.parametrize("over,code", [(dict(shares=FAKE + 2), 9), (dict(num_pages=-1), 3), (dict(num_pages=1 << 31), 3)])
def test_plan_refuses_bad_shares(over, code):
    a = M.kda_latent_plan_args(FAKE, FAKE, FAKE, 6, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 6, 8, 64, 100, FAKE, 10)
    assert _call("plan", _set(a, over)) == code
