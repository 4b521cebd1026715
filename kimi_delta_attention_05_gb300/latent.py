"""Python binding of the latent-attention calls (include/kda_latent.h): plan,
cache append, absorbed decode and expanded prefill.

Checks of types, shapes and strides happen here (ValueError), everything else
in the library (KdaError with its status code).  PyTorch supplies device memory
and the stream; buffers made here are allocated on the stream that uses them.
Page ids, lengths and slots are device values: what is wrong with them is read
from :func:`get_status`.
"""
from __future__ import annotations

import ctypes

import torch

from .kda import KdaError, load_library

LATENT_DIM = 512
LATENT_PE_DIM = 64
LATENT_ROW = LATENT_DIM + LATENT_PE_DIM
LATENT_QK_DIM = 192
LATENT_V_DIM = 128
KDA_LATENT_CAUSAL = 0x1

_P, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float


class kda_latent_plan_args(ctypes.Structure):
    _fields_ = [("cached_lens", _P), ("new_lens", _P), ("block_table", _P), ("table_stride", _I),
                ("free_pages", _P), ("seq_lens", _P), ("cu_seqlens", _P), ("slot_map", _P),
                ("pages_taken", _P), ("B", _I), ("max_pages", _I), ("num_free", _I),
                ("page_size", _I), ("T", _I)]


class kda_latent_cache(ctypes.Structure):
    _fields_ = [("data", _P), ("num_pages", _I), ("page_size", _I), ("page_stride", _I),
                ("token_stride", _I)]


class kda_latent_append_args(ctypes.Structure):
    _fields_ = [("c", _P), ("k_pe", _P), ("c_stride", _I), ("k_pe_stride", _I), ("slot_map", _P),
                ("cache", kda_latent_cache), ("norm_weight", _P), ("eps", _F), ("T", _I)]


class kda_latent_decode_args(ctypes.Structure):
    _fields_ = [("q", _P), ("cache", kda_latent_cache), ("block_table", _P), ("table_stride", _I),
                ("max_pages", _I), ("seq_lens", _P), ("scale", _F), ("out", _P), ("lse", _P),
                ("B", _I), ("R", _I), ("H", _I)]


class kda_latent_prefill_args(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("k_pe", _P), ("v", _P),
                ("q_stride_t", _I), ("q_stride_h", _I), ("k_stride_t", _I), ("k_stride_h", _I),
                ("k_pe_stride_t", _I), ("v_stride_t", _I), ("v_stride_h", _I), ("scale", _F),
                ("out", _P), ("lse", _P), ("cu_seqlens_q", _P), ("cu_seqlens_k", _P),
                ("B", _I), ("Tq", _I), ("Tk", _I), ("H", _I), ("N", _I), ("flags", ctypes.c_uint32)]


_fns = None


def _library():
    global _fns
    if _fns is None:
        lib = load_library()
        lib.kda_latent_plan.restype = ctypes.c_int
        lib.kda_latent_plan.argtypes = [ctypes.POINTER(kda_latent_plan_args), _P]
        lib.kda_latent_append.restype = ctypes.c_int
        lib.kda_latent_append.argtypes = [ctypes.POINTER(kda_latent_append_args), _P]
        for name, args in (("decode", kda_latent_decode_args), ("prefill", kda_latent_prefill_args)):
            fn = getattr(lib, f"kda_latent_{name}")
            fn.restype = ctypes.c_int
            fn.argtypes = [ctypes.POINTER(args), _P, ctypes.c_size_t, _P]
            size = getattr(lib, f"kda_latent_{name}_workspace_bytes")
            size.restype = ctypes.c_size_t
            size.argtypes = [ctypes.POINTER(args)]
        _fns = lib
    return _fns


def _raise(call, rc):
    raise KdaError(rc, _library().kda_error_string(rc).decode(), call)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _on(t, dtype, ndim, device, name):
    """A CUDA tensor of this type and rank on `device`."""
    if t.dtype is not dtype or t.dim() != ndim or t.device != device:
        raise ValueError(f"{name}: a {ndim}-d {dtype} tensor on {device} is needed, "
                         f"got {t.dim()}-d {t.dtype} on {t.device}")


def _rows(t, name):
    """Innermost dimension contiguous."""
    if t.stride(-1) != 1 and t.numel() > 0:
        raise ValueError(f"{name}: the last dimension has to be contiguous")


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is needed")


def _gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is needed, got one on {t.device}")
    return t.device


class _Call:
    """The stream of a call, and allocation on it.  The tensor's device has to
    be the current one, as for every launch of the library."""

    __slots__ = ("stream", "handle", "side")

    def __init__(self, device, stream):
        current = torch.cuda.current_stream(device)
        self.side = stream is not None and stream != current
        self.stream = stream if self.side else current
        self.handle = self.stream.cuda_stream

    def empty(self, shape, dtype, device):
        if not self.side:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=device)


def _cache_block(cache, device):
    _on(cache, torch.bfloat16, 3, device, "cache")
    _need(cache.shape[2] == LATENT_ROW, f"cache: rows of {LATENT_ROW} values are needed")
    _rows(cache, "cache")
    pages, page, _ = cache.shape
    token_stride = cache.stride(1)
    page_stride = cache.stride(0) if pages > 1 else (page - 1) * token_stride + LATENT_ROW + (-LATENT_ROW) % 8
    return kda_latent_cache(cache.data_ptr(), pages, page, page_stride, token_stride)


def latent_plan(cached_lens, new_lens, block_table, free_pages, page_size, num_tokens, *, stream=None):
    """Block tables and slot maps on the GPU from request lengths.

    cached_lens, new_lens int32 [B]; block_table int32 [B, max_pages], updated in
    place with pages taken from free_pages (int32) in order; ``num_tokens``: the
    capacity of the slot map (at least the sum of new_lens).  Returns a dict of
    device tensors: seq_lens int32 [B], cu_seqlens int64 [B + 1], slot_map int64
    [num_tokens] (-1 behind the last token), pages_taken int32 [1].  Lengths that
    do not fit, or too few free pages, plan nothing and show in
    :func:`get_status` (18 / 19)."""
    dev = _gpu(cached_lens, "cached_lens")
    for t, name in ((cached_lens, "cached_lens"), (new_lens, "new_lens"), (free_pages, "free_pages")):
        _on(t, torch.int32, 1, dev, name)
        _dense(t, name)
    _on(block_table, torch.int32, 2, dev, "block_table")
    _rows(block_table, "block_table")
    B = cached_lens.shape[0]
    _need(new_lens.shape[0] == B and block_table.shape[0] == B, "cached_lens, new_lens and block_table: one row a request")
    c = _Call(dev, stream)
    T, width = int(num_tokens), block_table.shape[1]
    lens = c.empty((B,), torch.int32, dev)
    cu = c.empty((B + 1,), torch.int64, dev)
    slots = c.empty((max(T, 0),), torch.int64, dev)
    taken = c.empty((1,), torch.int32, dev)
    a = kda_latent_plan_args(cached_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
                             block_table.stride(0) if B > 1 else width, free_pages.data_ptr(), lens.data_ptr(),
                             cu.data_ptr(), slots.data_ptr(), taken.data_ptr(), B, width, free_pages.shape[0],
                             int(page_size), T)
    rc = _library().kda_latent_plan(ctypes.byref(a), c.handle)
    if rc != 0:
        _raise("kda_latent_plan", rc)
    return {"seq_lens": lens, "cu_seqlens": cu, "slot_map": slots, "pages_taken": taken}


def latent_append(c, k_pe, slot_map, cache, norm_weight=None, eps=1e-6, *, stream=None):
    """Write new tokens' rows into the paged cache and return it.

    c bf16 [T, 512] and k_pe bf16 [T, 64] (views of one projection's output are
    fine), slot_map int64 [T] (negative: skipped), cache bf16 [pages, page_size,
    576]; norm_weight fp32 [512]: the latents are RMS-normalised with ``eps``
    and scaled on the way."""
    dev = _gpu(cache, "cache")
    _on(c, torch.bfloat16, 2, dev, "c")
    _on(k_pe, torch.bfloat16, 2, dev, "k_pe")
    _on(slot_map, torch.int64, 1, dev, "slot_map")
    T = c.shape[0]
    _need(c.shape[1] == LATENT_DIM and k_pe.shape[1] == LATENT_PE_DIM and k_pe.shape[0] == T and slot_map.shape[0] == T,
          "c [T, 512], k_pe [T, 64] and slot_map [T] are needed")
    _rows(c, "c")
    _rows(k_pe, "k_pe")
    _dense(slot_map, "slot_map")
    if norm_weight is not None:
        _on(norm_weight, torch.float32, 1, dev, "norm_weight")
        _need(norm_weight.shape[0] == LATENT_DIM, "norm_weight [512] is needed")
        _dense(norm_weight, "norm_weight")
    a = kda_latent_append_args(c.data_ptr(), k_pe.data_ptr(), c.stride(0) if T > 1 else LATENT_DIM,
                               k_pe.stride(0) if T > 1 else LATENT_PE_DIM, slot_map.data_ptr(),
                               _cache_block(cache, dev), None if norm_weight is None else norm_weight.data_ptr(),
                               float(eps), T)
    rc = _library().kda_latent_append(ctypes.byref(a), _Call(dev, stream).handle)
    if rc != 0:
        _raise("kda_latent_append", rc)
    return cache


def latent_decode(q, cache, block_table, seq_lens, scale, out=None, lse=None, *, workspace=None, stream=None):
    """Absorbed attention of every request's newest tokens over the paged cache;
    returns ``out``.

    q bf16 [B, R, H, 576] (R new tokens a request, whose rows the cache already
    holds), cache bf16 [pages, page_size, 576], block_table int32 [B, max_pages],
    seq_lens int32 [B]; out bf16 [B, R, H, 512] (allocated here if None), lse an
    optional fp32 [B, R, H] tensor to be written.  ``workspace``: an optional
    uint8 tensor of at least :func:`latent_decode_workspace_bytes` bytes."""
    dev = _gpu(q, "q")
    _on(q, torch.bfloat16, 4, dev, "q")
    B, R, H, D = q.shape
    _need(D == LATENT_ROW, f"q: heads of {LATENT_ROW} values are needed")
    _dense(q, "q")
    _on(block_table, torch.int32, 2, dev, "block_table")
    _rows(block_table, "block_table")
    _on(seq_lens, torch.int32, 1, dev, "seq_lens")
    _dense(seq_lens, "seq_lens")
    _need(block_table.shape[0] == B and seq_lens.shape[0] == B, "block_table and seq_lens: one row a request")
    c = _Call(dev, stream)
    if out is None:
        out = c.empty((B, R, H, LATENT_DIM), torch.bfloat16, dev)
    else:
        _on(out, torch.bfloat16, 4, dev, "out")
        _need(out.shape == (B, R, H, LATENT_DIM), "out [B, R, H, 512] is needed")
        _dense(out, "out")
    if lse is not None:
        _on(lse, torch.float32, 3, dev, "lse")
        _need(lse.shape == (B, R, H), "lse [B, R, H] is needed")
        _dense(lse, "lse")
    width = block_table.shape[1]
    a = kda_latent_decode_args(q.data_ptr(), _cache_block(cache, dev), block_table.data_ptr(),
                               block_table.stride(0) if B > 1 else width, width, seq_lens.data_ptr(), float(scale),
                               out.data_ptr(), None if lse is None else lse.data_ptr(), B, R, H)
    lib, ref = _library(), ctypes.byref(a)
    need = lib.kda_latent_decode_workspace_bytes(ref)
    if workspace is None and need:
        workspace = c.empty((need,), torch.uint8, dev)
    rc = lib.kda_latent_decode(ref, workspace.data_ptr() if workspace is not None else None,
                               workspace.numel() if workspace is not None else 0, c.handle)
    if rc != 0:
        _raise("kda_latent_decode", rc)
    return out


def latent_decode_workspace_bytes(B, R, H, cache, block_table):
    """Workspace bytes of :func:`latent_decode` for these sizes on the current device."""
    a = kda_latent_decode_args(16, _cache_block(cache, cache.device), 16, block_table.shape[1], block_table.shape[1], 16,
                               1.0, 16, None, B, R, H)
    return int(_library().kda_latent_decode_workspace_bytes(ctypes.byref(a)))


def _tokens(t, name, heads):
    """Token and head strides of a [B, T, H, .] (or [B, T, .]) tensor whose batch rows follow one another."""
    _rows(t, name)
    B, T = t.shape[0], t.shape[1]
    st = t.stride(1) if T > 1 else (t.stride(0) if B > 1 else None)
    if B > 1 and T > 0 and t.stride(0) != T * st:
        raise ValueError(f"{name}: batch rows have to follow one another")
    if not heads:
        return st if st is not None else t.shape[2]
    sh = t.stride(2) if t.shape[2] > 1 else t.shape[3]
    return (st if st is not None else max(sh * t.shape[2], t.shape[3])), sh


def latent_prefill(q, k, k_pe, v, scale, out=None, lse=None, cu_seqlens=None, cu_seqlens_k=None, *, causal=True,
                   workspace=None, stream=None):
    """Expanded attention of prompts; returns ``out``.

    q bf16 [B, Tq, H, 192], k bf16 [B, Tk, H, 128] (the heads' own key channels),
    k_pe bf16 [B, Tk, 64] (shared by the heads), v bf16 [B, Tk, H, 128]; k and v
    may be views of one up-projection's [.., H, 256] output.  cu_seqlens int64
    [N + 1] packs sequences (B == 1); cu_seqlens_k (default: cu_seqlens) gives
    the keys' own offsets where context precedes the queries.  Query i sees the
    keys j <= i + Lk - Lq, or all with ``causal=False``.  out bf16 [B, Tq, H,
    128]; lse an optional fp32 [B, Tq, H] tensor to be written."""
    dev = _gpu(q, "q")
    for t, d, name in ((q, 4, "q"), (k, 4, "k"), (k_pe, 3, "k_pe"), (v, 4, "v")):
        _on(t, torch.bfloat16, d, dev, name)
    B, Tq, H, D = q.shape
    Tk = k.shape[1]
    _need(D == LATENT_QK_DIM and k.shape == (B, Tk, H, 128) and v.shape == (B, Tk, H, LATENT_V_DIM)
          and k_pe.shape == (B, Tk, LATENT_PE_DIM),
          "q [B, Tq, H, 192], k and v [B, Tk, H, 128] and k_pe [B, Tk, 64] are needed")
    c = _Call(dev, stream)
    if out is None:
        out = c.empty((B, Tq, H, LATENT_V_DIM), torch.bfloat16, dev)
    else:
        _on(out, torch.bfloat16, 4, dev, "out")
        _need(out.shape == (B, Tq, H, LATENT_V_DIM), "out [B, Tq, H, 128] is needed")
        _dense(out, "out")
    if lse is not None:
        _on(lse, torch.float32, 3, dev, "lse")
        _need(lse.shape == (B, Tq, H), "lse [B, Tq, H] is needed")
        _dense(lse, "lse")
    N = B
    if cu_seqlens is not None:
        if cu_seqlens_k is None:
            cu_seqlens_k = cu_seqlens
        for t, name in ((cu_seqlens, "cu_seqlens"), (cu_seqlens_k, "cu_seqlens_k")):
            _on(t, torch.int64, 1, dev, name)
            _dense(t, name)
        N = cu_seqlens.shape[0] - 1
        _need(N >= 0 and cu_seqlens_k.shape[0] == N + 1, "cu_seqlens and cu_seqlens_k: [N + 1] each")
    else:
        _need(cu_seqlens_k is None, "cu_seqlens_k needs cu_seqlens")
    q_st, q_sh = _tokens(q, "q", True)
    k_st, k_sh = _tokens(k, "k", True)
    v_st, v_sh = _tokens(v, "v", True)
    a = kda_latent_prefill_args(
        q.data_ptr(), k.data_ptr(), k_pe.data_ptr(), v.data_ptr(), q_st, q_sh, k_st, k_sh,
        _tokens(k_pe, "k_pe", False), v_st, v_sh, float(scale), out.data_ptr(),
        None if lse is None else lse.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(),
        None if cu_seqlens is None else cu_seqlens_k.data_ptr(), B, Tq, Tk, H, N,
        KDA_LATENT_CAUSAL if causal else 0)
    lib, ref = _library(), ctypes.byref(a)
    need = lib.kda_latent_prefill_workspace_bytes(ref)
    if workspace is None and need:
        workspace = c.empty((need,), torch.uint8, dev)
    rc = lib.kda_latent_prefill(ref, workspace.data_ptr() if workspace is not None else None,
                                workspace.numel() if workspace is not None else 0, c.handle)
    if rc != 0:
        _raise("kda_latent_prefill", rc)
    return out
