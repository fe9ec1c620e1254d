"""Python binding of include/tsv_paged.h: rotary positions and the paged 8-bit KV cache.

Two layers, as in the package's main module: ``tsv_*`` functions mirror the C
ABI one to one; ``rope_frequencies``, ``rope``, ``PagedCache``, ``paged_append``,
``paged_tree_attention`` and ``paged_commit`` check shapes and types, allocate
what the caller did not pass, and call them.  The launches go to the current
stream of the tensors' device, or to ``stream``; what these helpers allocate
belongs to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import (TSV_ATTN_DEFAULT, TSV_BF16, TSV_F32, TSV_MAX_NODES, _check, _lib, _ptr, _workspace, handle)

PAGED_EXPORTED = (
    "tsv_rope_frequencies", "tsv_rope", "tsv_paged_append", "tsv_paged_tree_attention_workspace_size",
    "tsv_paged_tree_attention", "tsv_paged_commit",
)

TSV_ROPE_INTERLEAVED, TSV_ROPE_INVERSE = 1, 2
(TSV_ROPE_SCALE_NONE, TSV_ROPE_SCALE_LINEAR, TSV_ROPE_SCALE_NTK, TSV_ROPE_SCALE_BANDS,
 TSV_ROPE_SCALE_YARN) = range(5)
_SCALINGS = {"none": TSV_ROPE_SCALE_NONE, "linear": TSV_ROPE_SCALE_LINEAR, "ntk": TSV_ROPE_SCALE_NTK,
             "bands": TSV_ROPE_SCALE_BANDS, "yarn": TSV_ROPE_SCALE_YARN}


class CPagedCache(ctypes.Structure):
    """tsv_paged_cache."""
    _fields_ = [("k_d", ctypes.c_void_p), ("v_d", ctypes.c_void_p), ("k_scale_d", ctypes.c_void_p),
                ("v_scale_d", ctypes.c_void_p), ("stride_page", ctypes.c_int64), ("stride_row", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32)]


class CPageTable(ctypes.Structure):
    """tsv_page_table."""
    _fields_ = [("ids_d", ctypes.c_void_p), ("stride", ctypes.c_int64), ("pages", ctypes.c_int32)]


def _declare():
    vp, i32, i64, u32, f32, f64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                       ctypes.c_float, ctypes.c_double, ctypes.c_size_t)
    cache, table, e = ctypes.POINTER(CPagedCache), ctypes.POINTER(CPageTable), ctypes.c_int
    sig = {
        "tsv_rope_frequencies": [i32, f64, e, f64, f64, f64, f64, ctypes.POINTER(f64), ctypes.POINTER(f32)],
        "tsv_rope": [vp, e, vp, i64, i64, vp, i64, i64, i32, i32, i32, vp, vp, i32, f32, u32, vp],
        "tsv_paged_append": [vp, e, cache, table, vp, vp, i64, i64, vp, i64, i64, vp, i32, i32, i32, vp, vp, i32, f32,
                             u32, vp, vp],
        "tsv_paged_tree_attention_workspace_size": [vp, e, cache, i32, i32, i32, u32, ctypes.POINTER(sz)],
        "tsv_paged_tree_attention": [vp, e, vp, i64, i64, cache, table, vp, table, vp, vp, vp, i32, i32, i32, i32, f32,
                                     vp, sz, vp, u32, vp],
        "tsv_paged_commit": [vp, cache, table, table, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(_lib, name)
        f.restype, f.argtypes = ctypes.c_int, args


_declare()


# ----------------------------------------------------------------- C ABI mirror


def tsv_rope_frequencies(rotary_dim, base, scaling, factor, trained, low, high):
    """(list of rotary_dim / 2 frequencies, amplitude)."""
    out = (ctypes.c_double * max(int(rotary_dim) // 2, 1))()
    amplitude = ctypes.c_float()
    _check(_lib.tsv_rope_frequencies(int(rotary_dim), base, int(scaling), factor, trained, low, high, out,
                                     ctypes.byref(amplitude)), "tsv_rope_frequencies")
    return list(out), amplitude.value


def tsv_rope(h, dtype_code, x, x_stride_n, x_stride_h, y, y_stride_n, y_stride_h, N, H, D, positions, inv_freq,
             rotary_dim, amplitude, flags, stream):
    _check(_lib.tsv_rope(h, dtype_code, _ptr(x), x_stride_n, x_stride_h, _ptr(y), y_stride_n, y_stride_h, N, H, D,
                         _ptr(positions), _ptr(inv_freq), rotary_dim, amplitude, flags, stream), "tsv_rope")


def tsv_paged_append(h, dtype_code, cache, table, start, k, k_stride_n, k_stride_h, v, v_stride_n, v_stride_h,
                     row_offsets, B, N, max_rows, positions, inv_freq, rotary_dim, amplitude, flags, status, stream):
    """cache: CPagedCache, table: CPageTable."""
    _check(_lib.tsv_paged_append(h, dtype_code, cache, table, _ptr(start), _ptr(k), k_stride_n, k_stride_h, _ptr(v),
                                 v_stride_n, v_stride_h, _ptr(row_offsets), B, N, max_rows, _ptr(positions),
                                 _ptr(inv_freq), rotary_dim, amplitude, flags, _ptr(status), stream),
           "tsv_paged_append")


def tsv_paged_tree_attention_workspace_size(h, dtype_code, cache, B, max_nodes, Hq, flags=TSV_ATTN_DEFAULT) -> int:
    out = ctypes.c_size_t()
    _check(_lib.tsv_paged_tree_attention_workspace_size(h, dtype_code, cache, int(B), int(max_nodes), int(Hq), int(flags),
                                                        ctypes.byref(out)), "tsv_paged_tree_attention_workspace_size")
    return out.value


def tsv_paged_tree_attention(h, dtype_code, q, q_stride_n, q_stride_h, cache, table, prefix_len, tree_table,
                             node_offsets, anc, out, B, N, max_nodes, Hq, scale, workspace, workspace_bytes, status,
                             flags, stream):
    """tree_table: CPageTable or None."""
    _check(_lib.tsv_paged_tree_attention(h, dtype_code, _ptr(q), q_stride_n, q_stride_h, cache, table, _ptr(prefix_len),
                                         tree_table, _ptr(node_offsets), _ptr(anc), _ptr(out), B, N, max_nodes, Hq,
                                         scale, _ptr(workspace), workspace_bytes, _ptr(status), flags, stream),
           "tsv_paged_tree_attention")


def tsv_paged_commit(h, cache, table, tree_table, prefix_len, node_offsets, path, accept_len, B, N, max_nodes, new_len,
                     status, stream):
    _check(_lib.tsv_paged_commit(h, cache, table, tree_table, _ptr(prefix_len), _ptr(node_offsets), _ptr(path),
                                 _ptr(accept_len), B, N, max_nodes, _ptr(new_len), _ptr(status), stream),
           "tsv_paged_commit")


# ----------------------------------------------------------------- convenience layer


def _on(stream, dev):
    """The raw stream to launch on."""
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _allocating(stream, dev):
    """Context in which allocations belong to the stream that the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    s = torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream
    return torch.cuda.stream(s)


def _code(dt):
    if dt == torch.bfloat16:
        return TSV_BF16
    if dt == torch.float32:
        return TSV_F32
    raise TypeError("the paged cache's operators take bfloat16 or float32 rows, got %s" % dt)


def _want(ok, what):
    if not ok:
        raise ValueError(what)


def _ints(name, t, size, dev):
    """An int32 vector of `size` values on the call's device."""
    if t.dtype != torch.int32 or t.device != dev or t.dim() != 1 or t.shape[0] != size or not t.is_contiguous():
        raise ValueError("%s: a contiguous int32 tensor of %d values on %s is wanted" % (name, size, dev))


def _table(name, t, B, dev):
    if t.dtype != torch.int32 or t.device != dev or t.dim() != 2 or t.shape[0] != B or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s: an int32 tensor [%d, pages] on %s is wanted" % (name, B, dev))
    return CPageTable(t.data_ptr(), t.stride(0), t.shape[1])


def _heads(name, t, dev, D=None):
    """Rows of heads [N, H, D] with the elements of a head next to each other."""
    if t.device != dev or t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1 and t.numel()) or (D is not None and t.shape[2] != D):
        raise ValueError("%s: rows of heads [N, H, %s] on %s with contiguous heads are wanted"
                         % (name, "D" if D is None else D, dev))


def rope_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, trained=0.0, low=1.0, high=32.0, device=None):
    """Angular frequencies (float64 [rotary_dim / 2], on `device` when given) and the amplitude of a rotary position
    encoding.  `scaling`: "none", "linear", "ntk", "bands" or "yarn" (tsv_rope_scaling); `trained` is the context length
    the model was trained on, `low` and `high` the turns in it between which "bands" and "yarn" mix."""
    if scaling not in _SCALINGS:
        raise ValueError("scaling is one of %s" % ", ".join(_SCALINGS))
    f, amplitude = tsv_rope_frequencies(rotary_dim, float(base), _SCALINGS[scaling], float(factor), float(trained),
                                        float(low), float(high))
    return torch.tensor(f, dtype=torch.float64, device=device), amplitude


def _freqs(inv_freq, dev, D):
    if inv_freq.dtype != torch.float64 or inv_freq.device != dev or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq: a contiguous float64 vector on %s is wanted" % dev)
    rot = 2 * inv_freq.shape[0]
    _want(2 <= rot <= D, "inv_freq: 1 to D / 2 frequencies are wanted")
    return rot


def rope(x, positions, inv_freq, interleaved=False, inverse=False, amplitude=1.0, out=None, stream=None):
    """Rotates the first 2 * len(inv_freq) elements of every head of x [N, H, D] by its row's position; `inverse` turns
    back (the gradient of the rotation).  `out` may be x (in place).  Returns out."""
    dev = x.device
    _heads("x", x, dev)
    N, H, D = x.shape
    _ints("positions", positions, N, dev)
    rot = _freqs(inv_freq, dev, D)
    if out is None:
        with _allocating(stream, dev):
            out = torch.empty((N, H, D), dtype=x.dtype, device=dev)
    else:
        _heads("out", out, dev, D)
        _want(out.shape == x.shape and out.dtype == x.dtype, "out: x's shape and type are wanted")
    flags = (TSV_ROPE_INTERLEAVED if interleaved else 0) | (TSV_ROPE_INVERSE if inverse else 0)
    tsv_rope(handle(dev.index), _code(x.dtype), x, x.stride(0), x.stride(1), out, out.stride(0), out.stride(1), N, H, D,
             positions, inv_freq, rot, float(amplitude), flags, _on(stream, dev))
    return out


class PagedCache:
    """Pages of an 8-bit KV cache: k and v [num_pages, page_size, Hkv, D] (float8_e4m3fn, or uint8 holding its codes; any
    strides with d contiguous, the same for both) and k_scale, v_scale float32 [num_pages, Hkv]."""

    def __init__(self, k, v, k_scale, v_scale):
        kinds = (torch.float8_e4m3fn, torch.uint8)
        _want(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride() and k.stride(3) == 1,
              "k and v: [num_pages, page_size, Hkv, D] of equal strides with d contiguous are wanted")
        if k.dtype not in kinds or v.dtype not in kinds:
            raise TypeError("k and v hold 8-bit codes (float8_e4m3fn or uint8), got %s and %s" % (k.dtype, v.dtype))
        for s in (k_scale, v_scale):
            _want(s.dtype == torch.float32 and s.shape == (k.shape[0], k.shape[2]) and s.is_contiguous() and s.device == k.device,
                  "k_scale and v_scale: contiguous float32 [num_pages, Hkv] beside k are wanted")
        _want(k.device == v.device and k.device.type == "cuda", "k and v: tensors of one CUDA device are wanted")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.page_size, self.Hkv, self.D = k.shape
        self.device = k.device
        self.c = CPagedCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.stride(0), k.stride(1),
                             k.stride(2), *k.shape)

    @classmethod
    def empty(cls, num_pages, page_size, Hkv, D, device="cuda", head_major=True):
        """A cache of its own.  head_major: the rows of a head lie next to each other inside a page (one contiguous piece
        per page and head, what the attention reads); else the heads of a row do."""
        device = torch.empty(0, device=device).device
        shape = (num_pages, Hkv, page_size, D) if head_major else (num_pages, page_size, Hkv, D)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
        if head_major:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        ks, vs = (torch.zeros((num_pages, Hkv), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def paged_append(cache, page_table, k, v, row_offsets, start=None, positions=None, inv_freq=None, interleaved=False,
                 amplitude=1.0, max_rows=None, status=None, stream=None):
    """Writes rows row_offsets[b] .. row_offsets[b+1]-1 of k and v [N, Hkv, D] as rows start[b] .. of request b's pages
    (start None: from row 0), K rotated by `positions` when inv_freq is given; see tsv_paged_append for the scales.
    `max_rows`: the most new rows of one request (default N).  Returns status [B]."""
    dev = cache.device
    B = row_offsets.shape[0] - 1
    _heads("k", k, dev, cache.D)
    _heads("v", v, dev, cache.D)
    N = k.shape[0]
    _want(k.shape[1] == cache.Hkv and v.shape == k.shape and v.dtype == k.dtype, "k and v: [N, Hkv, D] of one type are wanted")
    _ints("row_offsets", row_offsets, B + 1, dev)
    rot = 0
    if inv_freq is not None:
        rot = _freqs(inv_freq, dev, cache.D)
        _want(positions is not None, "positions are wanted with inv_freq")
        _ints("positions", positions, N, dev)
    if start is not None:
        _ints("start", start, B, dev)
    if status is None:
        with _allocating(stream, dev):
            status = torch.empty(B, dtype=torch.int32, device=dev)
    else:
        _ints("status", status, B, dev)
    tsv_paged_append(handle(dev.index), _code(k.dtype), cache.c, _table("page_table", page_table, B, dev), start, k,
                     k.stride(0), k.stride(1), v, v.stride(0), v.stride(1), row_offsets, B, N,
                     N if max_rows is None else int(max_rows), positions if rot else None, inv_freq, rot, float(amplitude),
                     TSV_ROPE_INTERLEAVED if interleaved else 0, status, _on(stream, dev))
    return status


def paged_tree_attention_workspace(q, cache, B, max_nodes, flags=TSV_ATTN_DEFAULT):
    """A zero-filled workspace for calls of this shape, one at a time."""
    need = tsv_paged_tree_attention_workspace_size(handle(q.device.index), _code(q.dtype), cache.c, B, max_nodes, q.shape[1], flags)
    return _workspace(need, q.device)


def paged_tree_attention(q, cache, page_table, prefix_len, node_offsets, tree_table=None, anc=None, max_nodes=None,
                         scale=0.0, flags=TSV_ATTN_DEFAULT, out=None, workspace=None, status=None, stream=None):
    """Tree attention over the paged cache: q [N, Hq, D] -> out [N, Hq, D] and status [B].  prefix_len, node_offsets and
    both page tables are device tensors; anc [N, 8] comes from tree_prepare (None: a chain of new tokens); tree_table
    None: the nodes see the prefix alone.  `max_nodes`: the most nodes of one request (default min(N, 256))."""
    dev = cache.device
    B = node_offsets.shape[0] - 1
    _heads("q", q, dev, cache.D)
    N, Hq, D = q.shape
    _ints("prefix_len", prefix_len, B, dev)
    _ints("node_offsets", node_offsets, B + 1, dev)
    if anc is not None:
        _want(anc.dtype == torch.int32 and anc.device == dev and anc.shape == (N, 8) and anc.is_contiguous(),
              "anc: the contiguous int32 [N, 8] of tree_prepare is wanted")
    if max_nodes is None:
        max_nodes = max(1, min(N, TSV_MAX_NODES))
    h = handle(dev.index)
    code = _code(q.dtype)
    with _allocating(stream, dev):
        if out is None:
            out = torch.empty((N, Hq, D), dtype=q.dtype, device=dev)
        else:
            _want(out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous() and out.device == dev,
                  "out: a contiguous tensor of q's shape and type is wanted")
        if status is None:
            status = torch.empty(B, dtype=torch.int32, device=dev)
        else:
            _ints("status", status, B, dev)
        if workspace is None:
            workspace = _workspace(tsv_paged_tree_attention_workspace_size(h, code, cache.c, B, max_nodes, Hq, flags), dev)
    tsv_paged_tree_attention(h, code, q, q.stride(0), q.stride(1), cache.c, _table("page_table", page_table, B, dev),
                             prefix_len, None if tree_table is None else _table("tree_table", tree_table, B, dev),
                             node_offsets, anc, out, B, N, int(max_nodes), Hq, float(scale), workspace, workspace.numel(),
                             status, int(flags), _on(stream, dev))
    return out, status


def paged_commit(cache, page_table, tree_table, prefix_len, node_offsets, path, accept_len, max_nodes=None, stream=None,
                 out=None):
    """Appends the accepted path's rows of the tree pages to the prefix pages: row prefix_len[b] + k takes tree row
    path[k].  Returns dict(new_len, status)."""
    dev = cache.device
    B = node_offsets.shape[0] - 1
    N = path.shape[0]
    _ints("prefix_len", prefix_len, B, dev)
    _ints("node_offsets", node_offsets, B + 1, dev)
    _ints("path", path, N, dev)
    _ints("accept_len", accept_len, B, dev)
    if out is None:
        with _allocating(stream, dev):
            out = dict(new_len=torch.empty(B, dtype=torch.int32, device=dev),
                       status=torch.empty(B, dtype=torch.int32, device=dev))
    else:
        _ints("new_len", out["new_len"], B, dev)
        _ints("status", out["status"], B, dev)
    tsv_paged_commit(handle(dev.index), cache.c, _table("page_table", page_table, B, dev),
                     _table("tree_table", tree_table, B, dev), prefix_len, node_offsets, path, accept_len, B, N,
                     max(1, min(N, TSV_MAX_NODES)) if max_nodes is None else int(max_nodes), out["new_len"], out["status"],
                     _on(stream, dev))
    return out
