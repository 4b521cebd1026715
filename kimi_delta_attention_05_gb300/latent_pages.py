"""Python binding of the calls for cache pages that several requests hold
(include/kda_latent.h): fork, release, compact and copy.

``shares`` int32 [num_pages] counts the holders of a page beyond the first: it
starts as zeros, and pages taken by :func:`latent_plan` are right as they come.
Checks, streams, devices and errors are those of :mod:`.latent`; request numbers,
lengths and page ids are device values: what is wrong with them is read from
:func:`get_status`.
"""
from __future__ import annotations

import ctypes

import torch

from .latent import (_I, _P, _cache_block, _dense, _gpu, _handle, _i32, _last, _library, _new, _on, _packer, _raise,
                     kda_latent_cache)


class kda_latent_fork_args(ctypes.Structure):
    _fields_ = [("parents", _P), ("children", _P), ("fork_lens", _P), ("cached_lens", _P), ("block_table", _P),
                ("table_stride", _I), ("free_pages", _P), ("shares", _P), ("cache", kda_latent_cache),
                ("seq_lens", _P), ("pages_taken", _P), ("F", _I), ("B", _I), ("max_pages", _I), ("num_free", _I)]


class kda_latent_release_args(ctypes.Structure):
    _fields_ = [("rows", _P), ("keep_lens", _P), ("cached_lens", _P), ("block_table", _P), ("table_stride", _I),
                ("shares", _P), ("seq_lens", _P), ("pages", _P), ("count", _P), ("F", _I), ("B", _I),
                ("max_pages", _I), ("num_pages", _I), ("page_size", _I)]


class kda_latent_compact_args(ctypes.Structure):
    _fields_ = [("cached_lens", _P), ("block_table", _P), ("table_stride", _I), ("block_table_out", _P),
                ("table_out_stride", _I), ("shares", _P), ("shares_out", _P), ("page_map", _P), ("pages_used", _P),
                ("cache", kda_latent_cache), ("B", _I), ("max_pages", _I)]


class kda_latent_copy_args(ctypes.Structure):
    _fields_ = [("src", kda_latent_cache), ("dst", kda_latent_cache), ("src_pages", _P), ("dst_pages", _P), ("n", _I)]


_empty_like = torch.empty_like
_fork_block, _release_block = _packer(kda_latent_fork_args), _packer(kda_latent_release_args)
_compact_block, _copy_block = _packer(kda_latent_compact_args), _packer(kda_latent_copy_args)


def _ints(t, device, name):
    """Address and length of a contiguous int32 vector."""
    if t.dtype is not _i32 or t.ndim != 1 or t.device != device or not t.is_contiguous():
        _on(t, _i32, 1, device, name)
        _dense(t, name)
    return t.data_ptr(), t.shape[0]


def _like(t, stream):
    """Memory as large as t, dense, allocated on the stream that uses it."""
    if stream is None and t.is_contiguous():
        return _empty_like(t)  # (a fifth faster than a call with sizes, type and device)
    return _new(t.shape, t.dtype, t.device, stream)


def _requests(cached_lens, block_table, stream):
    """Device, lengths' address, and address, stride, rows and width of the table of a call."""
    dev = _gpu(cached_lens, "cached_lens", stream)
    lens, n = _ints(cached_lens, dev, "cached_lens")
    table, stride, B, width = _table(block_table, dev, "block_table")
    if n != B:
        raise ValueError("cached_lens and block_table: one row a request")
    return dev, lens, table, stride, B, width


def _table(t, device, name):
    """Address, stride, rows and width of a table."""
    if t.dtype is not _i32 or t.ndim != 2 or t.device != device:
        _on(t, _i32, 2, device, name)
    B, width = t.shape
    strides = t.stride()
    if strides[1] != 1:
        _last(strides, t, name)
    return t.data_ptr(), strides[0] if B > 1 else width, B, width


def latent_fork(parents, children, cached_lens, block_table, free_pages, shares, cache, fork_lens=None, *, stream=None):
    """Requests that go on from other requests' tokens.

    Request ``children[f]`` gets the first ``fork_lens[f]`` tokens (default: all) of
    request ``parents[f]`` (int32 [F] each): whole pages are shared, the rows of a last
    page that is not whole are copied to the next page of free_pages.  block_table
    int32 [B, max_pages], shares int32 [num_pages] and cache are updated in place.
    No child twice, as a parent or with tokens: what its row held before has to be
    released first.  Returns a dict of device tensors: seq_lens int32 [B] and pages_taken
    int32 [1].  Numbers and lengths that do not fit, or too few free pages, fork
    nothing and show in :func:`get_status` (18 / 19)."""
    dev, lens, table, stride, B, width = _requests(cached_lens, block_table, stream)
    of, F = _ints(parents, dev, "parents")
    to, n = _ints(children, dev, "children")
    if n != F:
        raise ValueError("parents and children: one entry a fork")
    take = 0
    if fork_lens is not None:
        take, n = _ints(fork_lens, dev, "fork_lens")
        if n != F:
            raise ValueError("fork_lens: one entry a fork")
    free, num_free = _ints(free_pages, dev, "free_pages")
    block = _cache_block(cache, dev)
    counts, n = _ints(shares, dev, "shares")
    if n != block[1]:
        raise ValueError("shares: one entry a page of the cache")
    out = _like(cached_lens, stream)
    taken = _new(1, _i32, dev, stream)
    a = _fork_block(of, to, take, lens, table, stride, free, counts, *block, out.data_ptr(), taken.data_ptr(), F, B, width,
                    num_free)
    rc = _library().kda_latent_fork(a, _handle(dev, stream))
    if rc != 0:
        _raise("kda_latent_fork", rc)
    return {"seq_lens": out, "pages_taken": taken}


def latent_release(rows, cached_lens, block_table, shares, page_size, keep_lens=None, *, stream=None):
    """Requests that give pages back: ``rows`` (int32 [F], none twice) keep their first
    ``keep_lens`` tokens (int32 [F]; default: none) and drop the pages behind them.

    block_table int32 [B, max_pages] stays as it is; shares int32 [num_pages] is
    updated in place.  Returns a dict of device tensors: seq_lens int32 [B], pages
    int32 [num_pages] (those that nobody holds any more, ascending, and -1 behind
    them) and count int32 [1].  Rows and lengths that do not fit release nothing
    and show in :func:`get_status` (18).  A row that keeps part of a page that others
    hold must not grow from there (:func:`latent_plan` refuses it where it is given
    shares; :func:`latent_fork` with fork_lens copies that part)."""
    dev, lens, table, stride, B, width = _requests(cached_lens, block_table, stream)
    at, F = _ints(rows, dev, "rows")
    keep = 0
    if keep_lens is not None:
        keep, n = _ints(keep_lens, dev, "keep_lens")
        if n != F:
            raise ValueError("keep_lens: one entry a row")
    counts, num_pages = _ints(shares, dev, "shares")
    out = _like(cached_lens, stream)
    pages = _like(shares, stream)
    count = _new(1, _i32, dev, stream)
    a = _release_block(at, keep, lens, table, stride, counts, out.data_ptr(), pages.data_ptr(), count.data_ptr(), F, B, width,
                       num_pages, int(page_size))
    rc = _library().kda_latent_release(a, _handle(dev, stream))
    if rc != 0:
        _raise("kda_latent_release", rc)
    return {"seq_lens": out, "pages": pages, "count": count}


def latent_compact(cached_lens, block_table, shares, cache, *, out_table=None, out_shares=None, stream=None):
    """Held pages together: of the U pages that the table's rows hold, those with ids
    from U on move to the places below that nobody holds, in ascending order.

    Rows move within ``cache``.  Returns a dict of device tensors: block_table and
    shares by the new ids (new tensors, or ``out_table`` and ``out_shares``, which may
    be the inputs), page_map int32 [num_pages] (new id of every held page, -1 for
    others) and pages_used int32 [1], U: pages U and behind are free.  Lengths that do
    not fit move nothing and show in :func:`get_status` (18)."""
    dev, lens, table, stride, B, width = _requests(cached_lens, block_table, stream)
    block = _cache_block(cache, dev)
    pages = block[1]
    counts, n = _ints(shares, dev, "shares")
    if n != pages:
        raise ValueError("shares: one entry a page of the cache")
    if out_table is None:
        out_table = _like(block_table, stream)
    to, to_stride, rows, columns = _table(out_table, dev, "out_table")
    if (rows, columns) != (B, width):
        raise ValueError("out_table: as large as block_table")
    if to == table and to_stride != stride:
        raise ValueError("out_table: another view of block_table's memory")
    if out_shares is None:
        out_shares = _like(shares, stream)
    to_counts, n = _ints(out_shares, dev, "out_shares")
    if n != pages:
        raise ValueError("out_shares: one entry a page of the cache")
    page_map = _like(shares, stream)
    used = _new(1, _i32, dev, stream)
    a = _compact_block(lens, table, stride, to, to_stride, counts, to_counts, page_map.data_ptr(), used.data_ptr(), *block, B,
                       width)
    rc = _library().kda_latent_compact(a, _handle(dev, stream))
    if rc != 0:
        _raise("kda_latent_compact", rc)
    return {"block_table": out_table, "shares": out_shares, "page_map": page_map, "pages_used": used}


def latent_copy(src, src_pages, dst, dst_pages, *, stream=None):
    """Copy pages ``src_pages`` of cache ``src`` into pages ``dst_pages`` (int32 [n],
    distinct) of cache ``dst``, which is returned; both caches bf16 [pages, page_size,
    576], strides may differ.  They may be the same tensor where no page is both read
    and written."""
    dev = _gpu(dst, "dst", stream)
    at, n = _ints(src_pages, dev, "src_pages")
    to, m = _ints(dst_pages, dev, "dst_pages")
    if n != m:
        raise ValueError("src_pages and dst_pages: one entry a page")
    rc = _library().kda_latent_copy(_copy_block(*_cache_block(src, dev), *_cache_block(dst, dev), at, to, n),
                                    _handle(dev, stream))
    if rc != 0:
        _raise("kda_latent_copy", rc)
    return dst
