"""Python binding of include/tsv_pages.h: which request holds which page of a paged cache.

Two layers, as in the package's main module: ``tsv_pages_*`` mirror the C ABI one to one; ``PagePool``, ``pages_resize``,
``pages_fork``, ``pages_compact`` and ``pages_copy`` check shapes and types, allocate what the caller did not pass, and call
them.  The launches go to the current stream of the tensors' device, or to ``stream``; what these helpers allocate belongs to
that stream.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _check, _lib, _ptr
from .paged import CPagedCache, CPageTable, _allocating, _at, _handle, _ints, _on, _table, _want

PAGES_EXPORTED = ("tsv_pages_resize", "tsv_pages_fork", "tsv_pages_compact", "tsv_pages_copy")

TSV_PAGES_MAX_LISTS = 8


class CPagePool(ctypes.Structure):
    """tsv_page_pool."""
    _fields_ = [("refs_d", ctypes.c_void_p), ("num_pages", ctypes.c_int32)]


class CPageLists(ctypes.Structure):
    """tsv_page_lists."""
    _fields_ = [("table", CPageTable), ("pages_d", ctypes.c_void_p), ("out_d", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("B", ctypes.c_int32)]


def _declare():
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    sig = {
        "tsv_pages_resize": [vp, vp, vp, vp, vp, i32, i32, vp, vp],
        "tsv_pages_fork": [vp, vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp],
        "tsv_pages_compact": [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp],
        "tsv_pages_copy": [vp, vp, vp, vp, i32, vp, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(_lib, name)
        f.restype, f.argtypes = ctypes.c_int, args


_declare()


# ----------------------------------------------------------------- C ABI mirror


def tsv_pages_resize(h, pool, table, pages, rows, B, page_size, status, stream):
    """pool: CPagePool, table: CPageTable."""
    _check(_lib.tsv_pages_resize(h, _at(pool), _at(table), _ptr(pages), _ptr(rows), B, page_size, _ptr(status), stream),
           "tsv_pages_resize")


def tsv_pages_fork(h, pool, from_table, from_pages, F, source, rows, to_table, to_pages, B, page_size, copy_src, copy_dst, status,
                   stream):
    _check(_lib.tsv_pages_fork(h, _at(pool), _at(from_table), _ptr(from_pages), F, _ptr(source), _ptr(rows), _at(to_table),
                               _ptr(to_pages), B, page_size, _ptr(copy_src), _ptr(copy_dst), _ptr(status), stream),
           "tsv_pages_fork")


def tsv_pages_compact(h, pool, refs_out, lists, n, new_id, move_src, move_dst, moved, status, stream):
    """lists: an array of CPageLists."""
    _check(_lib.tsv_pages_compact(h, _at(pool), _ptr(refs_out), None if lists is None else ctypes.addressof(lists), n, _ptr(new_id),
                                  _ptr(move_src), _ptr(move_dst), _ptr(moved), _ptr(status), stream), "tsv_pages_compact")


def tsv_pages_copy(h, cache, src, dst, n, count, status, stream):
    """cache: CPagedCache."""
    _check(_lib.tsv_pages_copy(h, _at(cache), _ptr(src), _ptr(dst), n, _ptr(count), _ptr(status), stream), "tsv_pages_copy")


# ----------------------------------------------------------------- convenience layer


_INT = torch.int32
_pack_lists = struct.Struct("@Pqi4xPPqi4x").pack  # CPageLists' bytes
assert struct.calcsize("@Pqi4xPPqi4x") == ctypes.sizeof(CPageLists)


class PagePool:
    """Reference counts of a cache's pages: `refs` int32 [num_pages], 0 for a free page.  PagePool(num_pages) makes one with
    every page free; PagePool(refs) takes over a tensor of counts."""

    def __init__(self, pages, device="cuda"):
        if not isinstance(pages, torch.Tensor):
            pages = torch.zeros(pages, dtype=_INT, device=device)
        _want(pages.dtype is _INT and pages.dim() == 1 and pages.is_contiguous() and pages.device.type == "cuda" and len(pages) > 0,
              "refs: a contiguous int32 vector on a CUDA device is wanted")
        self.refs = pages
        self.num_pages = pages.shape[0]
        self.device = pages.device
        self.index = pages.get_device()
        self.c = CPagePool(pages.data_ptr(), self.num_pages)
        self.at = ctypes.addressof(self.c)


def _empty(pool, stream, *sizes):
    with _allocating(stream, pool.device):
        return [torch.empty(n, dtype=_INT, device=pool.device) for n in sizes]


def pages_resize(pool, page_table, pages, rows, page_size, status=None, stream=None):
    """Request b's list (row b of page_table, pages[b] entries held) gets the pages of rows[b] rows: what is too much goes back
    to the pool, what lacks comes from it, lowest ids first.  page_table, pages and the pool change in place.  Returns
    status [B]."""
    index = pool.index
    B = page_table.shape[0]
    table = _table("page_table", page_table, B, index)
    held, want = _ints("pages", pages, B, index), _ints("rows", rows, B, index)
    if status is None:
        status, = _empty(pool, stream, B)
    st = _ints("status", status, B, index)
    _check(_lib.tsv_pages_resize(_handle(index), pool.at, table, held, want, B, page_size, st, _on(stream, index)),
           "tsv_pages_resize")
    return status


def pages_fork(pool, from_table, from_pages, source, rows, to_table, to_pages, page_size, out=None, stream=None):
    """List b of to_table becomes the first rows[b] rows of list source[b] of from_table (source -1: stays as it is): whole
    pages are shared, a partly filled last one gets a page of its own.  What list b held goes back to the pool.  to_table,
    to_pages and the pool change in place.  Returns dict(copy_src, copy_dst, status), each [B]; in every layer's cache
    pages_copy(cache, copy_src, copy_dst) follows."""
    index = pool.index
    F, B = from_table.shape[0], to_table.shape[0]
    first, second = _table("from_table", from_table, F, index), _table("to_table", to_table, B, index)
    has, held = _ints("from_pages", from_pages, F, index), _ints("to_pages", to_pages, B, index)
    src, want = _ints("source", source, B, index), _ints("rows", rows, B, index)
    if out is None:
        out = dict(zip(("copy_src", "copy_dst", "status"), _empty(pool, stream, B, B, B)))
    a, b, st = (_ints(name, out[name], B, index) for name in ("copy_src", "copy_dst", "status"))
    _check(_lib.tsv_pages_fork(_handle(index), pool.at, first, has, F, src, want, second, held, B, page_size, a, b, st,
                               _on(stream, index)), "tsv_pages_fork")
    return out


def pages_compact(pool, tables, pages, out=None, in_place=False, stream=None):
    """The pages in use move to the lowest ids.  `tables`, `pages`: every list of the pool, as up to 8 page tables [B, width] and
    their counts [B].  Returns dict(refs, tables, new_id, move_src, move_dst, moved, status): the counts and tables under the
    new ids (in place: the pool's and the tables' own), the new id of every page, and the `moved` [1] pages that change theirs;
    in every layer's cache pages_copy(cache, move_src, move_dst, count=moved) follows.  Entries of a table behind its counts
    are not written."""
    index, P, n = pool.index, pool.num_pages, len(tables)
    _want(len(pages) == n <= TSV_PAGES_MAX_LISTS, "tables and pages: up to %d of each are wanted" % TSV_PAGES_MAX_LISTS)
    if out is None:
        new_id, src, dst, moved, status = _empty(pool, stream, P, P // 2 + 1, P // 2 + 1, 1, n)
        out = dict(new_id=new_id, move_src=src, move_dst=dst, moved=moved, status=status, refs=pool.refs, tables=list(tables))
        if not in_place:
            out["refs"], = _empty(pool, stream, P)
            with _allocating(stream, pool.device):
                out["tables"] = [torch.empty(t.shape, dtype=_INT, device=pool.device) for t in tables]
    elif "status" not in out:
        out = dict(out, status=_empty(pool, stream, n)[0])
    _want(len(out["tables"]) == n, "out: as many tables are wanted")
    packed = b""
    for i, (t, held, to) in enumerate(zip(tables, pages, out["tables"])):
        shape, ts, os = t.shape, t.stride(), to.stride()
        if (t.dtype is not _INT or to.dtype is not _INT or t.get_device() != index or to.get_device() != index or len(shape) != 2
                or to.shape != shape or (shape[1] > 1 and not ts[1] == os[1] == 1)):
            raise ValueError("tables[%d]: int32 tensors [B, pages] of one shape on cuda:%d are wanted, the new one too" % (i, index))
        B, width = shape
        packed += _pack_lists(t.data_ptr(), ts[0], width, _ints("pages", held, B, index), to.data_ptr(), os[0], B)
    refs, ids = _ints("refs", out["refs"], P, index), _ints("new_id", out["new_id"], P, index)
    src, dst = out["move_src"], out["move_dst"]
    room, room_dst = src.numel(), dst.numel()
    _want(room >= P // 2 and room_dst >= P // 2, "move_src and move_dst: half the pool's pages of room are wanted")
    a, b = _ints("move_src", src, room, index), _ints("move_dst", dst, room_dst, index)
    count, st = _ints("moved", out["moved"], 1, index), _ints("status", out["status"], n, index)
    _check(_lib.tsv_pages_compact(_handle(index), pool.at, refs, packed or None, n, ids, a, b, count, st, _on(stream, index)),
           "tsv_pages_compact")
    return out


def pages_copy(cache, src, dst, count=None, status=None, stream=None):
    """Page dst[i] of the cache takes the codes and scales of page src[i] (pairs with a -1 are left out); `count` [1] on the
    device: only the first so many pairs.  Returns status [1]."""
    index = cache.index
    n = src.shape[0]
    a, b = _ints("src", src, n, index), _ints("dst", dst, n, index)
    first = None if count is None else _ints("count", count, 1, index)
    if status is None:
        with _allocating(stream, cache.device):
            status = torch.empty(1, dtype=_INT, device=cache.device)
    st = _ints("status", status, 1, index)
    _check(_lib.tsv_pages_copy(_handle(index), cache.at, a, b, n, first, st, _on(stream, index)), "tsv_pages_copy")
    return status
