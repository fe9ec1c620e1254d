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
import struct

import torch

from . import TSV_ATTN_DEFAULT, TSV_BF16, TSV_F32, TSV_MAX_NODES, _HANDLES, _check, _lib, _ptr, _workspace, handle

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
    cache = table = vp  # structures go by their address: the quickest argument to convert
    e = ctypes.c_int
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


def _at(struct):
    """The address of a structure (None: NULL)."""
    return None if struct is None else ctypes.addressof(struct)


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
    _check(_lib.tsv_paged_append(h, dtype_code, _at(cache), _at(table), _ptr(start), _ptr(k), k_stride_n, k_stride_h, _ptr(v),
                                 v_stride_n, v_stride_h, _ptr(row_offsets), B, N, max_rows, _ptr(positions),
                                 _ptr(inv_freq), rotary_dim, amplitude, flags, _ptr(status), stream),
           "tsv_paged_append")


def tsv_paged_tree_attention_workspace_size(h, dtype_code, cache, B, max_nodes, Hq, flags=TSV_ATTN_DEFAULT) -> int:
    out = ctypes.c_size_t()
    _check(_lib.tsv_paged_tree_attention_workspace_size(h, dtype_code, _at(cache), int(B), int(max_nodes), int(Hq), int(flags),
                                                        ctypes.byref(out)), "tsv_paged_tree_attention_workspace_size")
    return out.value


def tsv_paged_tree_attention(h, dtype_code, q, q_stride_n, q_stride_h, cache, table, prefix_len, tree_table,
                             node_offsets, anc, out, B, N, max_nodes, Hq, scale, workspace, workspace_bytes, status,
                             flags, stream):
    """tree_table: CPageTable or None."""
    _check(_lib.tsv_paged_tree_attention(h, dtype_code, _ptr(q), q_stride_n, q_stride_h, _at(cache), _at(table),
                                         _ptr(prefix_len), _at(tree_table), _ptr(node_offsets), _ptr(anc), _ptr(out), B, N, max_nodes, Hq,
                                         scale, _ptr(workspace), workspace_bytes, _ptr(status), flags, stream),
           "tsv_paged_tree_attention")


def tsv_paged_commit(h, cache, table, tree_table, prefix_len, node_offsets, path, accept_len, B, N, max_nodes, new_len,
                     status, stream):
    _check(_lib.tsv_paged_commit(h, _at(cache), _at(table), _at(tree_table), _ptr(prefix_len), _ptr(node_offsets), _ptr(path),
                                 _ptr(accept_len), B, N, max_nodes, _ptr(new_len), _ptr(status), stream),
           "tsv_paged_commit")


# ----------------------------------------------------------------- convenience layer


_raw_stream = torch._C._cuda_getCurrentRawStream


def _on(stream, index):
    """The raw stream to launch on."""
    if stream is None:
        return _raw_stream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _allocating(stream, dev):
    """Context in which allocations belong to the stream that the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    s = torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream
    return torch.cuda.stream(s)


_CODES = {torch.bfloat16: TSV_BF16, torch.float32: TSV_F32}
_INT = torch.int32


def _code(dt):
    code = _CODES.get(dt)
    if code is None:
        raise TypeError("the paged cache's operators take bfloat16 or float32 rows, got %s" % dt)
    return code


def _handle(index):
    h = _HANDLES.get(index)
    if h is None:
        with torch.cuda.device(index):  # (tsv_create makes the device current)
            h = handle(index)
    return h


def _want(ok, what):
    if not ok:
        raise ValueError(what)


def _ints(name, t, size, index):
    """The address of an int32 vector of `size` values on the call's device."""
    if t.dtype is not _INT or t.get_device() != index or t.shape != (size,) or not t.is_contiguous():
        raise ValueError("%s: a contiguous int32 tensor of %d values on cuda:%d is wanted" % (name, size, index))
    return t.data_ptr()


_pack_table = struct.Struct("@Pqi4x").pack  # CPageTable's bytes: made in a third of the structure's time
assert struct.calcsize("@Pqi4x") == ctypes.sizeof(CPageTable)


def _table(name, t, B, index):
    """A tsv_page_table, as its bytes."""
    if t.dtype is not _INT or t.get_device() != index or t.dim() != 2:
        raise ValueError("%s: an int32 tensor [%d, pages] on cuda:%d is wanted" % (name, B, index))
    rows, pages = t.shape
    stride, inner = t.stride()
    if rows != B or (pages > 1 and inner != 1) or pages >= 1 << 31:
        raise ValueError("%s: an int32 tensor [%d, pages] on cuda:%d is wanted" % (name, B, index))
    return _pack_table(t.data_ptr(), stride, pages)


def _heads(name, t, index, D=None):
    """Shape and strides of rows of heads [N, H, D] with the elements of a head next to each other."""
    if t.get_device() != index or t.dim() != 3:
        raise ValueError("%s: rows of heads [N, H, D] on cuda:%d are wanted" % (name, index))
    shape, strides = t.shape, t.stride()
    if (strides[2] != 1 and shape[2] > 1 and t.numel()) or (D is not None and shape[2] != D):
        raise ValueError("%s: rows of heads [N, H, %s] with contiguous heads are wanted" % (name, "D" if D is None else D))
    return shape, strides


def rope_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, trained=0.0, low=1.0, high=32.0, device=None):
    """Angular frequencies (float64 [rotary_dim / 2], on `device` when given) and the amplitude of a rotary position
    encoding.  `scaling`: "none", "linear", "ntk", "bands" or "yarn" (tsv_rope_scaling); `trained` is the context length
    the model was trained on, `low` and `high` the turns in it between which "bands" and "yarn" mix."""
    if scaling not in _SCALINGS:
        raise ValueError("scaling is one of %s" % ", ".join(_SCALINGS))
    f, amplitude = tsv_rope_frequencies(rotary_dim, float(base), _SCALINGS[scaling], float(factor), float(trained),
                                        float(low), float(high))
    return torch.tensor(f, dtype=torch.float64, device=device), amplitude


def _freqs(inv_freq, index, D):
    if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != index or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq: a contiguous float64 vector on cuda:%d is wanted" % index)
    rot = 2 * inv_freq.numel()
    _want(2 <= rot <= D, "inv_freq: 1 to D / 2 frequencies are wanted")
    return rot


def rope(x, positions, inv_freq, interleaved=False, inverse=False, amplitude=1.0, out=None, stream=None):
    """Rotates the first 2 * len(inv_freq) elements of every head of x [N, H, D] by its row's position; `inverse` turns
    back (the gradient of the rotation).  `out` may be x (in place).  Returns out."""
    index = x.get_device()
    shape, xs = _heads("x", x, index)
    _want(index >= 0, "x: a CUDA tensor is wanted")
    N, H, D = shape
    pos = _ints("positions", positions, N, index)
    rot = _freqs(inv_freq, index, D)
    code = _code(x.dtype)
    if out is None:
        with _allocating(stream, x.device):
            out = torch.empty((N, H, D), dtype=x.dtype, device=x.device)
        ys = out.stride()
    else:
        oshape, ys = _heads("out", out, index)
        _want(oshape == shape and out.dtype is x.dtype, "out: x's shape and type are wanted")
    flags = (TSV_ROPE_INTERLEAVED if interleaved else 0) | (TSV_ROPE_INVERSE if inverse else 0)
    _check(_lib.tsv_rope(_handle(index), code, x.data_ptr(), xs[0], xs[1], out.data_ptr(), ys[0], ys[1], N, H, D, pos,
                         inv_freq.data_ptr(), rot, amplitude, flags, _on(stream, index)), "tsv_rope")
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
        self.index = k.get_device()
        self.c = CPagedCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.stride(0), k.stride(1),
                             k.stride(2), *k.shape)
        self.at = ctypes.addressof(self.c)

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
    index = cache.index
    B = row_offsets.shape[0] - 1
    shape, ks = _heads("k", k, index, cache.D)
    vshape, vs = _heads("v", v, index)
    N = shape[0]
    _want(shape[1] == cache.Hkv and vshape == shape and v.dtype is k.dtype, "k and v: [N, Hkv, D] of one type are wanted")
    offs = _ints("row_offsets", row_offsets, B + 1, index)
    rot, pos, freq = 0, None, None
    if inv_freq is not None:
        rot, freq = _freqs(inv_freq, index, cache.D), inv_freq.data_ptr()
        _want(positions is not None, "positions are wanted with inv_freq")
        pos = _ints("positions", positions, N, index)
    first = None if start is None else _ints("start", start, B, index)
    table = _table("page_table", page_table, B, index)
    code = _code(k.dtype)
    if status is None:
        with _allocating(stream, cache.device):
            status = torch.empty(B, dtype=_INT, device=cache.device)
    st = _ints("status", status, B, index)
    _check(_lib.tsv_paged_append(_handle(index), code, cache.at, table, first, k.data_ptr(), ks[0], ks[1],
                                 v.data_ptr(), vs[0], vs[1], offs, B, N, N if max_rows is None else max_rows, pos, freq, rot,
                                 amplitude, TSV_ROPE_INTERLEAVED if interleaved else 0, st, _on(stream, index)),
           "tsv_paged_append")
    return status


def paged_tree_attention_workspace(q, cache, B, max_nodes, flags=TSV_ATTN_DEFAULT):
    """A zero-filled workspace for calls of this shape, one at a time."""
    need = tsv_paged_tree_attention_workspace_size(_handle(q.device.index), _code(q.dtype), cache.c, B, max_nodes, q.shape[1], flags)
    return _workspace(need, q.device)


def paged_tree_attention(q, cache, page_table, prefix_len, node_offsets, tree_table=None, anc=None, max_nodes=None,
                         scale=0.0, flags=TSV_ATTN_DEFAULT, out=None, workspace=None, status=None, stream=None):
    """Tree attention over the paged cache: q [N, Hq, D] -> out [N, Hq, D] and status [B].  prefix_len, node_offsets and
    both page tables are device tensors; anc [N, 8] comes from tree_prepare (None: a chain of new tokens); tree_table
    None: the nodes see the prefix alone.  `max_nodes`: the most nodes of one request (default min(N, 256))."""
    index = cache.index
    B = node_offsets.shape[0] - 1
    shape, qs = _heads("q", q, index, cache.D)
    N, Hq, D = shape
    plen = _ints("prefix_len", prefix_len, B, index)
    offs = _ints("node_offsets", node_offsets, B + 1, index)
    words = None
    if anc is not None:
        _want(anc.dtype is _INT and anc.get_device() == index and anc.shape == (N, 8) and anc.is_contiguous(),
              "anc: the contiguous int32 [N, 8] of tree_prepare is wanted")
        words = anc.data_ptr()
    if max_nodes is None:
        max_nodes = max(1, min(N, TSV_MAX_NODES))
    main = _table("page_table", page_table, B, index)
    tree = None if tree_table is None else _table("tree_table", tree_table, B, index)
    h, code = _handle(index), _code(q.dtype)
    if out is None or status is None or workspace is None:
        with _allocating(stream, cache.device):
            if out is None:
                out = torch.empty((N, Hq, D), dtype=q.dtype, device=cache.device)
            if status is None:
                status = torch.empty(B, dtype=_INT, device=cache.device)
            if workspace is None:
                workspace = _workspace(tsv_paged_tree_attention_workspace_size(h, code, cache.c, B, max_nodes, Hq, flags),
                                       cache.device)
    _want(out.shape == shape and out.dtype is q.dtype and out.is_contiguous() and out.get_device() == index,
          "out: a contiguous tensor of q's shape and type is wanted")
    _want(workspace.get_device() == index and workspace.is_contiguous(), "workspace: a contiguous tensor beside the cache is wanted")
    st = _ints("status", status, B, index)
    _check(_lib.tsv_paged_tree_attention(h, code, q.data_ptr(), qs[0], qs[1], cache.at, main, plen,
                                         tree, offs, words, out.data_ptr(), B, N,
                                         max_nodes, Hq, scale, workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), st, flags, _on(stream, index)),
           "tsv_paged_tree_attention")
    return out, status


def paged_commit(cache, page_table, tree_table, prefix_len, node_offsets, path, accept_len, max_nodes=None, stream=None,
                 out=None):
    """Appends the accepted path's rows of the tree pages to the prefix pages: row prefix_len[b] + k takes tree row
    path[k].  Returns dict(new_len, status)."""
    index = cache.index
    B = node_offsets.shape[0] - 1
    N = path.shape[0]
    plen = _ints("prefix_len", prefix_len, B, index)
    offs = _ints("node_offsets", node_offsets, B + 1, index)
    way = _ints("path", path, N, index)
    acc = _ints("accept_len", accept_len, B, index)
    main, tree = _table("page_table", page_table, B, index), _table("tree_table", tree_table, B, index)
    if out is None:
        with _allocating(stream, cache.device):
            out = dict(new_len=torch.empty(B, dtype=_INT, device=cache.device),
                       status=torch.empty(B, dtype=_INT, device=cache.device))
    new, st = _ints("new_len", out["new_len"], B, index), _ints("status", out["status"], B, index)
    _check(_lib.tsv_paged_commit(_handle(index), cache.at, main, tree, plen, offs, way, acc,
                                 B, N, max(1, min(N, TSV_MAX_NODES)) if max_nodes is None else max_nodes, new, st,
                                 _on(stream, index)), "tsv_paged_commit")
    return out
