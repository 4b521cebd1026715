"""Python binding of the latent-attention calls (include/kda_latent.h): plan,
cache append, absorbed decode and expanded prefill.

Checks of types, shapes and strides happen here (ValueError), everything else
in the library (KdaError with its status code).  PyTorch supplies device memory
and the stream; buffers made here are allocated on the stream that uses them.  Tensors and
stream have to be on the current device (ValueError otherwise).
Page ids, lengths and slots are device values: what is wrong with them is read
from :func:`get_status`.
"""
from __future__ import annotations

import ctypes
import struct

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


def _packer(block):
    """Packs the fields of an argument block, nested ones in place, into its bytes: one call
    where filling the ctypes structure takes three times as long."""
    # (a float beyond 32 bits goes in as infinity, _F(x).value, for the library to refuse: struct would raise its own error)
    codes = {_P: "P", _I: "q", _F: "f", ctypes.c_uint32: "I"}

    def fields(cls):
        return "".join(codes[t] if t in codes else fields(t) for _, t in cls._fields_)

    layout = struct.Struct("@" + fields(block) + "0q")
    assert layout.size == ctypes.sizeof(block)
    return layout.pack


_plan_block, _append_block = _packer(kda_latent_plan_args), _packer(kda_latent_append_args)
_decode_block, _prefill_block = _packer(kda_latent_decode_args), _packer(kda_latent_prefill_args)

_fns = None


def _library():
    global _fns
    if _fns is None:
        lib = load_library()
        for name in ("plan", "append", "decode", "prefill"):
            fn = getattr(lib, f"kda_latent_{name}")
            fn.restype = ctypes.c_int
            if name in ("plan", "append"):  # the block (its bytes or a reference), the stream
                fn.argtypes = [_P, _P]
                continue
            fn.argtypes = [_P, _P, ctypes.c_size_t, _P]
            size = getattr(lib, f"kda_latent_{name}_workspace_bytes")
            size.restype = ctypes.c_size_t
            size.argtypes = [_P]
        _fns = lib
    return _fns


_bf16, _f32, _i32, _i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_empty = torch.empty


def _raise(call, rc):
    raise KdaError(rc, _library().kda_error_string(rc).decode(), call)


# A serving step makes these calls every few microseconds: the checks are plain
# comparisons, and the messages are put together only on failure.

def _on(t, dtype, ndim, device, name):
    """A CUDA tensor of this type and rank on `device`."""
    if t.dtype is not dtype or t.ndim != ndim or t.device != device:
        raise ValueError(f"{name}: a {ndim}-d {dtype} tensor on {device} is needed, "
                         f"got {t.dim()}-d {t.dtype} on {t.device}")


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is needed")


# The current device's index without the checks around it, where this PyTorch has the call.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _gpu(t, name, stream):
    """The device of a call: the library sizes, launches and keeps its status words on the
    current device, so tensors and stream have to be of that one."""
    dev = t.device
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is needed, got one on {dev}")
    if dev.index != _current_device():
        raise ValueError(f"{name}: on {dev}, but the current device is cuda:{_current_device()} (torch.cuda.device sets it)")
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream: one of {dev} is needed, got one of {stream.device}")
    return dev


def _last(strides, t, name):
    if strides[-1] != 1 and t.shape[-1] > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the last dimension has to be contiguous")


def _scratch(workspace, device):
    """Address and bytes of a workspace."""
    if workspace is None:
        return None, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on {device} is needed, got one on {workspace.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# The handle of the current stream without the Stream object around it, where
# this PyTorch has the call (2 us less on the host).
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(device, stream):
    if stream is not None:
        return stream.cuda_stream
    if _current is not None:
        return _current(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _new(shape, dtype, device, stream):
    """Memory allocated on the stream that uses it."""
    if stream is None:
        return _empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return _empty(shape, dtype=dtype, device=device)


def _cache_block(cache, device):
    _on(cache, _bf16, 3, device, "cache")
    pages, page, row = cache.shape
    strides = cache.stride()
    if row != LATENT_ROW:
        raise ValueError(f"cache: rows of {LATENT_ROW} values are needed")
    _last(strides, cache, "cache")
    page_stride = strides[0] if pages > 1 else (page - 1) * strides[1] + LATENT_ROW
    return cache.data_ptr(), pages, page, page_stride, strides[1]


def latent_plan(cached_lens, new_lens, block_table, free_pages, page_size, num_tokens, *, stream=None):
    """Block tables and slot maps on the GPU from request lengths.

    cached_lens, new_lens int32 [B]; block_table int32 [B, max_pages], updated in
    place with pages taken from free_pages (int32) in order; ``num_tokens``: the
    capacity of the slot map (at least the sum of new_lens).  Returns a dict of
    device tensors: seq_lens int32 [B], cu_seqlens int64 [B + 1], slot_map int64
    [num_tokens] (-1 behind the last token), pages_taken int32 [1].  Lengths that
    do not fit, or too few free pages, plan nothing and show in
    :func:`get_status` (18 / 19)."""
    dev = _gpu(cached_lens, "cached_lens", stream)
    _on(cached_lens, _i32, 1, dev, "cached_lens")
    _on(new_lens, _i32, 1, dev, "new_lens")
    _on(free_pages, _i32, 1, dev, "free_pages")
    _on(block_table, _i32, 2, dev, "block_table")
    if not (cached_lens.is_contiguous() and new_lens.is_contiguous() and free_pages.is_contiguous()):
        raise ValueError("cached_lens, new_lens and free_pages: contiguous tensors are needed")
    B, width = block_table.shape
    strides = block_table.stride()
    _last(strides, block_table, "block_table")
    if cached_lens.shape[0] != B or new_lens.shape[0] != B:
        raise ValueError("cached_lens, new_lens and block_table: one row a request")
    T = int(num_tokens)
    lens = _new(B, _i32, dev, stream)
    cu = _new(B + 1, _i64, dev, stream)
    slots = _new(max(T, 0), _i64, dev, stream)
    taken = _new(1, _i32, dev, stream)
    a = _plan_block(cached_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), strides[0] if B > 1 else width,
                    free_pages.data_ptr(), lens.data_ptr(), cu.data_ptr(), slots.data_ptr(), taken.data_ptr(), B, width,
                    free_pages.shape[0], int(page_size), T)
    rc = _library().kda_latent_plan(a, _handle(dev, stream))
    if rc != 0:
        _raise("kda_latent_plan", rc)
    return {"seq_lens": lens, "cu_seqlens": cu, "slot_map": slots, "pages_taken": taken}


def latent_append(c, k_pe, slot_map, cache, norm_weight=None, eps=1e-6, *, stream=None):
    """Write new tokens' rows into the paged cache and return it.

    c bf16 [T, 512] and k_pe bf16 [T, 64] (views of one projection's output are
    fine), slot_map int64 [T] (negative: skipped), cache bf16 [pages, page_size,
    576]; norm_weight fp32 [512]: the latents are RMS-normalised with ``eps``
    and scaled on the way."""
    dev = _gpu(cache, "cache", stream)
    _on(c, _bf16, 2, dev, "c")
    _on(k_pe, _bf16, 2, dev, "k_pe")
    _on(slot_map, _i64, 1, dev, "slot_map")
    T, width = c.shape
    if width != LATENT_DIM or k_pe.shape != (T, LATENT_PE_DIM) or slot_map.shape[0] != T:
        raise ValueError("c [T, 512], k_pe [T, 64] and slot_map [T] are needed")
    c_strides, pe_strides = c.stride(), k_pe.stride()
    _last(c_strides, c, "c")
    _last(pe_strides, k_pe, "k_pe")
    _dense(slot_map, "slot_map")
    if norm_weight is not None:
        _on(norm_weight, _f32, 1, dev, "norm_weight")
        _dense(norm_weight, "norm_weight")
        if norm_weight.shape[0] != LATENT_DIM:
            raise ValueError("norm_weight [512] is needed")
    a = _append_block(c.data_ptr(), k_pe.data_ptr(), c_strides[0] if T > 1 else LATENT_DIM,
                      pe_strides[0] if T > 1 else LATENT_PE_DIM, slot_map.data_ptr(), *_cache_block(cache, dev),
                      0 if norm_weight is None else norm_weight.data_ptr(), _F(eps).value, T)
    rc = _library().kda_latent_append(a, _handle(dev, stream))
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
    dev = _gpu(q, "q", stream)
    _on(q, _bf16, 4, dev, "q")
    B, R, H, D = q.shape
    if D != LATENT_ROW:
        raise ValueError(f"q: heads of {LATENT_ROW} values are needed")
    _dense(q, "q")
    _on(block_table, _i32, 2, dev, "block_table")
    rows, width = block_table.shape
    strides = block_table.stride()
    _last(strides, block_table, "block_table")
    _on(seq_lens, _i32, 1, dev, "seq_lens")
    _dense(seq_lens, "seq_lens")
    if rows != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens: one row a request")
    if out is None:
        out = _new((B, R, H, LATENT_DIM), _bf16, dev, stream)
    else:
        _on(out, _bf16, 4, dev, "out")
        _dense(out, "out")
        if out.shape != (B, R, H, LATENT_DIM):
            raise ValueError("out [B, R, H, 512] is needed")
    if lse is not None:
        _on(lse, _f32, 3, dev, "lse")
        _dense(lse, "lse")
        if lse.shape != (B, R, H):
            raise ValueError("lse [B, R, H] is needed")
    a = _decode_block(q.data_ptr(), *_cache_block(cache, dev), block_table.data_ptr(), strides[0] if B > 1 else width,
                      width, seq_lens.data_ptr(), _F(scale).value, out.data_ptr(), 0 if lse is None else lse.data_ptr(), B, R, H)
    lib = _library()
    if workspace is None:
        need = lib.kda_latent_decode_workspace_bytes(a)
        workspace = _new(need, torch.uint8, dev, stream) if need else None
    rc = lib.kda_latent_decode(a, *_scratch(workspace, dev), _handle(dev, stream))
    if rc != 0:
        _raise("kda_latent_decode", rc)
    return out


def latent_decode_workspace_bytes(B, R, H, cache, block_table):
    """Workspace bytes of :func:`latent_decode` for these sizes on the current device."""
    width = block_table.shape[1]
    return int(_library().kda_latent_decode_workspace_bytes(
        _decode_block(16, *_cache_block(cache, cache.device), 16, width, width, 16, 1.0, 16, 0, B, R, H)))


def _token_stride(shape, strides, row, name):
    """Token stride of a [B, T, ...] tensor whose batch rows follow one another; `row` where it has one token."""
    B, T = shape[0], shape[1]
    if B > 1:
        if T > 1 and strides[0] != T * strides[1]:
            raise ValueError(f"{name}: batch rows have to follow one another")
        return strides[0] if T == 1 else strides[1]
    return strides[1] if T > 1 else row


_SPLIT_KEYS = 4096  # KDA_LATENT_SPLIT_KEYS: dense calls with fewer keys need no workspace, so it is not asked for


def latent_prefill(q, k, k_pe, v, scale, out=None, lse=None, cu_seqlens=None, cu_seqlens_k=None, *, causal=True,
                   workspace=None, stream=None):
    """Expanded attention of prompts; returns ``out``.

    q bf16 [B, Tq, H, 192], k bf16 [B, Tk, H, 128] (the heads' own key channels),
    k_pe bf16 [B, Tk, 64] (shared by the heads), v bf16 [B, Tk, H, 128]; k and v
    may be views of one up-projection's [.., H, 256] output.  cu_seqlens int64
    [N + 1] packs sequences (B == 1); cu_seqlens_k (default: cu_seqlens) gives
    the keys' own offsets where context precedes the queries.  Query i sees the
    keys j <= i + Lk - Lq, or all with ``causal=False``.  out bf16 [B, Tq, H,
    128]; lse an optional fp32 [B, Tq, H] tensor to be written.  ``workspace``: an
    optional uint8 tensor of at least :func:`latent_prefill_workspace_bytes` bytes."""
    dev = _gpu(q, "q", stream)
    _on(q, _bf16, 4, dev, "q")
    _on(k, _bf16, 4, dev, "k")
    _on(k_pe, _bf16, 3, dev, "k_pe")
    _on(v, _bf16, 4, dev, "v")
    B, Tq, H, D = shape = q.shape
    k_shape = k.shape
    Tk = k_shape[1]
    if (D != LATENT_QK_DIM or k_shape != (B, Tk, H, 128) or v.shape != k_shape
            or k_pe.shape != (B, Tk, LATENT_PE_DIM)):
        raise ValueError("q [B, Tq, H, 192], k and v [B, Tk, H, 128] and k_pe [B, Tk, 64] are needed")
    qs, ks, ps, vs = q.stride(), k.stride(), k_pe.stride(), v.stride()
    _last(qs, q, "q")
    _last(ks, k, "k")
    _last(ps, k_pe, "k_pe")
    _last(vs, v, "v")
    if out is None:
        out = _new((B, Tq, H, LATENT_V_DIM), _bf16, dev, stream)
    else:
        _on(out, _bf16, 4, dev, "out")
        _dense(out, "out")
        if out.shape != (B, Tq, H, LATENT_V_DIM):
            raise ValueError("out [B, Tq, H, 128] is needed")
    if lse is not None:
        _on(lse, _f32, 3, dev, "lse")
        _dense(lse, "lse")
        if lse.shape != (B, Tq, H):
            raise ValueError("lse [B, Tq, H] is needed")
    N, cu_q, cu_k = B, 0, 0
    if cu_seqlens is not None:
        if cu_seqlens_k is None:
            cu_seqlens_k = cu_seqlens
        _on(cu_seqlens, _i64, 1, dev, "cu_seqlens")
        _on(cu_seqlens_k, _i64, 1, dev, "cu_seqlens_k")
        _dense(cu_seqlens, "cu_seqlens")
        _dense(cu_seqlens_k, "cu_seqlens_k")
        N = cu_seqlens.shape[0] - 1
        if N < 0 or cu_seqlens_k.shape[0] != N + 1:
            raise ValueError("cu_seqlens and cu_seqlens_k: [N + 1] each")
        cu_q, cu_k = cu_seqlens.data_ptr(), cu_seqlens_k.data_ptr()
    elif cu_seqlens_k is not None:
        raise ValueError("cu_seqlens_k needs cu_seqlens")
    # (a dimension of one has no stride of its own)
    qh, kh, vh = (qs[2], ks[2], vs[2]) if H > 1 else (LATENT_QK_DIM, 128, LATENT_V_DIM)
    a = _prefill_block(
        q.data_ptr(), k.data_ptr(), k_pe.data_ptr(), v.data_ptr(), _token_stride(shape, qs, H * qh, "q"), qh,
        _token_stride(k_shape, ks, H * kh, "k"), kh, _token_stride(k_shape, ps, LATENT_PE_DIM, "k_pe"),
        _token_stride(k_shape, vs, H * vh, "v"), vh, _F(scale).value, out.data_ptr(), 0 if lse is None else lse.data_ptr(),
        cu_q, cu_k, B, Tq, Tk, H, N, KDA_LATENT_CAUSAL if causal else 0)
    lib = _library()
    if workspace is None and (cu_seqlens is not None or Tk >= _SPLIT_KEYS):
        need = lib.kda_latent_prefill_workspace_bytes(a)
        workspace = _new(need, torch.uint8, dev, stream) if need else None
    rc = lib.kda_latent_prefill(a, *_scratch(workspace, dev), _handle(dev, stream))
    if rc != 0:
        _raise("kda_latent_prefill", rc)
    return out


def latent_prefill_workspace_bytes(B, Tq, Tk, H, sequences=None, *, causal=True):
    """Workspace bytes of :func:`latent_prefill` for these sizes on the current device; ``sequences``: how many are packed."""
    cu = 0 if sequences is None else 16
    return int(_library().kda_latent_prefill_workspace_bytes(_prefill_block(
        16, 16, 16, 16, LATENT_QK_DIM * H, LATENT_QK_DIM, 128 * H, 128, LATENT_PE_DIM, 128 * H, 128, 1.0, 16, 0, cu, cu,
        B, Tq, Tk, H, B if sequences is None else sequences, KDA_LATENT_CAUSAL if causal else 0)))
