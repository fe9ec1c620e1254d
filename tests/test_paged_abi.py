"""include/tsv_paged.h: exports, binding, host-side refusals (no device needed)."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tsv_paged.h")


@pytest.fixture(scope="module")
def paged():
    import importlib.util
    spec = importlib.util.spec_from_file_location("tsv_build", os.path.join(
        ROOT, "tree_speculative_verification_attention_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.build()
    import tree_speculative_verification_attention_gb300 as tsv
    return tsv.paged


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_exports_binding_and_constants(paged):
    names = set(re.findall(r"^tsv_status\s+(tsv_[a-z_]+)\s*\(", _text(), re.M))
    assert names == set(paged.PAGED_EXPORTED)
    for n in names:
        assert hasattr(paged._lib, n) and callable(getattr(paged, n))
    found = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define\s+(TSV_[A-Z_]+)\s+(\d+)u", _text())}
    found.update({m.group(1): int(m.group(2)) for m in re.finditer(r"(TSV_ROPE_SCALE_[A-Z]+)\s*=\s*(\d+)", _text())})
    assert len(found) == 7
    for n, v in found.items():
        assert getattr(paged, n) == v


def test_header_is_plain_c_and_structs_match_the_binding(paged, tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tsv_paged.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu", sizeof(tsv_paged_cache), offsetof(tsv_paged_cache, stride_page), '
                   'offsetof(tsv_paged_cache, D), sizeof(tsv_page_table), offsetof(tsv_page_table, pages));\nreturn 0; }\n')
    exe = tmp_path / "t"
    cc = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I" + os.path.join(ROOT, "include"),
                         str(src), "-o", str(exe)], capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    C, T = paged.CPagedCache, paged.CPageTable
    assert got == [ctypes.sizeof(C), C.stride_page.offset, C.D.offset, ctypes.sizeof(T), T.pages.offset]


# ------------------------------------------------------------------ refusals
# A block of zeros stands for a handle and made-up addresses for buffers: a refused call touches neither.

HANDLE = ctypes.create_string_buffer(4096)
H = ctypes.cast(HANDLE, ctypes.c_void_p)
P = 1 << 20  # a 16-byte aligned address that nobody reads


def _cache(paged, **kw):
    f = dict(k_d=P, v_d=P, k_scale_d=P, v_scale_d=P, stride_page=16 * 2 * 64, stride_row=64, stride_head=16 * 64, num_pages=8,
             page_size=16, Hkv=2, D=64)
    f.update(kw)
    return paged.CPagedCache(**f)


def _table(paged, **kw):
    f = dict(ids_d=P, stride=4, pages=4)
    f.update(kw)
    return paged.CPageTable(**f)


def _call(paged, name, **kw):
    cache = kw.pop("cache", _cache(paged))
    table, tree = kw.pop("table", _table(paged)), kw.pop("tree", _table(paged))
    orders = {
        "tsv_rope": dict(h=H, dtype=1, x=P, xn=128, xh=64, y=P + 64, yn=128, yh=64, N=3, H=2, D=64, pos=P, freq=P, rot=64,
                         amp=1.0, flags=0, stream=None),
        "tsv_paged_append": dict(h=H, dtype=1, cache=cache, table=table, start=P, k=P, kn=128, kh=64, v=P, vn=128, vh=64,
                                 offs=P, B=2, N=5, max_rows=5, pos=P, freq=P, rot=64, amp=1.0, flags=0, status=P, stream=None),
        "tsv_paged_tree_attention": dict(h=H, dtype=1, q=P, qn=256, qh=64, cache=cache, table=table, plen=P, tree=tree, offs=P,
                                         anc=P, out=P, B=2, N=5, max_nodes=4, Hq=4, scale=0.0, ws=P, wsb=1 << 40, status=P,
                                         flags=0, stream=None),
        "tsv_paged_commit": dict(h=H, cache=cache, table=table, tree=tree, plen=P, offs=P, path=P, acc=P, B=2, N=5,
                                 max_nodes=4, new=P + 64, status=P, stream=None),
    }
    args = orders[name]
    for k in kw:
        assert k in args, k
    args.update(kw)
    return _raw(paged, name, *args.values())


def _raw(paged, name, *args):
    """The C function, structures by their address."""
    return getattr(paged._lib, name)(*[paged._at(x) if isinstance(x, ctypes.Structure) else x for x in args])


BAD = {
    "tsv_rope": [dict(h=None), dict(dtype=2), dict(flags=4), dict(N=-1), dict(H=0), dict(D=1), dict(rot=0), dict(rot=3),
                 dict(rot=66), dict(x=None), dict(y=None), dict(pos=None), dict(freq=None), dict(y=P, yn=64)],
    "tsv_paged_append": [dict(h=None), dict(dtype=7), dict(flags=2), dict(B=0), dict(B=129), dict(N=-1), dict(max_rows=-1),
                         dict(offs=None), dict(status=None), dict(k=None), dict(v=None), dict(pos=None), dict(rot=0),
                         dict(rot=66), dict(rot=7), dict(k=P + 8), dict(vn=4), dict(kh=12)],
    "tsv_paged_tree_attention": [dict(h=None), dict(dtype=-1), dict(flags=2), dict(B=0), dict(B=129), dict(max_nodes=0),
                                 dict(max_nodes=257), dict(Hq=0), dict(Hq=3), dict(plen=None), dict(offs=None),
                                 dict(status=None), dict(N=-1), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
                                 dict(anc=P + 4), dict(q=None), dict(out=None), dict(out=P + 8), dict(qn=4), dict(qh=2)],
    "tsv_paged_commit": [dict(h=None), dict(B=0), dict(B=129), dict(N=-1), dict(max_nodes=0), dict(max_nodes=257),
                         dict(plen=None), dict(offs=None), dict(path=None), dict(acc=None), dict(status=None), dict(new=P)],
}


@pytest.mark.parametrize("name", sorted(BAD))
def test_bad_arguments_are_refused(paged, name):
    for kw in BAD[name]:
        assert _call(paged, name, **kw) == 1, (name, kw)


@pytest.mark.parametrize("name", ["tsv_paged_append", "tsv_paged_tree_attention", "tsv_paged_commit"])
def test_bad_caches_and_tables_are_refused(paged, name):
    for kw in (dict(k_d=None), dict(v_d=P + 8), dict(k_scale_d=None), dict(v_scale_d=P + 2), dict(num_pages=0), dict(Hkv=0),
               dict(stride_row=0), dict(stride_row=72), dict(stride_head=-64), dict(stride_page=8)):
        assert _call(paged, name, cache=_cache(paged, **kw)) == 1, kw
    for kw in (dict(D=96), dict(page_size=8), dict(page_size=48), dict(num_pages=1 << 28)):
        assert _call(paged, name, cache=_cache(paged, **kw)) == 3, kw
    for kw in (dict(ids_d=None), dict(pages=0), dict(stride=3)):
        assert _call(paged, name, table=_table(paged, **kw)) == 1, kw
        if name != "tsv_paged_append":
            assert _call(paged, name, tree=_table(paged, **kw)) == 1, kw
    dtype = [] if name == "tsv_paged_commit" else [1]
    assert _raw(paged, name, H, *dtype, *_nulls(paged, name)) == 1


def _nulls(paged, name):
    """The call with NULL in the place of the cache."""
    t = _table(paged)
    return {"tsv_paged_append": [None, t, P, P, 128, 64, P, 128, 64, P, 2, 5, 5, P, P, 64, 1.0, 0, P, None],
            "tsv_paged_tree_attention": [P, 256, 64, None, t, P, t, P, P, P, 2, 5, 4, 4, 0.0, P, 0, P, 0, None],
            "tsv_paged_commit": [None, t, t, P, P, P, P, 2, 5, 4, P + 64, P, None]}[name]


def test_good_arguments_reach_the_device(paged):
    """The arguments that the refusals above start from are accepted: what stops them here is that there is no device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present: the made-up addresses must not reach it")
    for name in BAD:
        assert _call(paged, name) == 4, name


def test_workspace_size_refusals(paged):
    n = ctypes.c_size_t(7)
    f = lambda *a: _raw(paged, "tsv_paged_tree_attention_workspace_size", *a)  # noqa: E731
    c = _cache(paged)
    assert f(None, 1, c, 1, 1, 4, 0, ctypes.byref(n)) == 1
    assert f(H, 1, c, 1, 1, 4, 0, None) == 1
    assert f(H, 1, c, 1, 1, 3, 0, ctypes.byref(n)) == 1
    assert f(H, 1, _cache(paged, D=32), 1, 1, 4, 0, ctypes.byref(n)) == 3
    assert n.value == 7


# ------------------------------------------------------------------ frequencies (host arithmetic)


def test_frequencies(paged):
    f = lambda *a: np.array(paged.tsv_rope_frequencies(*a)[0])  # noqa: E731
    i = np.arange(64)
    plain = 10000.0 ** (-2.0 * i / 128)
    assert np.allclose(f(128, 1e4, 0, 0, 0, 0, 0), plain, rtol=1e-14)
    assert np.allclose(f(128, 1e4, 1, 4.0, 0, 0, 0), plain / 4, rtol=1e-14)
    assert np.allclose(f(128, 1e4, 2, 4.0, 0, 0, 0), (1e4 * 4 ** (128 / 126)) ** (-2.0 * i / 128), rtol=1e-13)
    turns = 8192 * plain / (2 * math.pi)
    keep = np.clip((turns - 1) / 3, 0, 1)
    assert np.allclose(f(128, 1e4, 3, 8.0, 8192.0, 1.0, 4.0), plain * keep + plain / 8 * (1 - keep), rtol=1e-13)
    w, amp = paged.tsv_rope_frequencies(128, 1e4, 4, 4.0, 4096.0, 1.0, 32.0)
    at = lambda t: 128 * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(1e4))  # noqa: E731
    lo, hi = math.floor(at(32.0)), math.ceil(at(1.0))
    keep = 1 - np.clip((i - lo) / (hi - lo), 0, 1)
    assert np.allclose(w, plain * keep + plain / 4 * (1 - keep), rtol=1e-13)
    assert abs(amp - (0.1 * math.log(4) + 1)) < 1e-6
    assert np.allclose(f(2, 1e4, 2, 4.0, 0, 0, 0), [1.0])


def test_frequencies_refusals(paged):
    out, amp = (ctypes.c_double * 64)(), ctypes.c_float()
    f = paged._lib.tsv_rope_frequencies
    good = [128, 1e4, 4, 4.0, 4096.0, 1.0, 32.0, out, ctypes.byref(amp)]
    assert f(*good) == 0
    for i, x in ((0, 0), (0, 3), (1, 0.0), (1, math.inf), (1, math.nan), (1, 1.0), (2, 5), (2, -1), (3, 0.0), (3, math.inf),
                 (4, 0.0), (5, 0.0), (6, 0.5), (6, math.inf), (7, None), (8, None)):
        bad = list(good)
        bad[i] = x
        assert f(*bad) == 1, (i, x)


# ------------------------------------------------------------------ devices


def test_the_first_call_on_a_device_leaves_the_current_one(paged, monkeypatch):
    """A handle that a call makes (tsv_create makes its device current) does not change the caller's device."""
    from types import SimpleNamespace

    now = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *error):
            now[0] = self.before

    def create(index):
        now[0] = index
        return 7

    monkeypatch.setattr(paged.torch.cuda, "device", Device)
    monkeypatch.setattr(paged, "_HANDLES", {})
    monkeypatch.setattr(paged, "handle", create)
    assert paged._handle(1) == 7 and now == [0]
    monkeypatch.setattr(paged, "tsv_paged_tree_attention_workspace_size", lambda h, *shape: 16 if h == 7 else None)
    monkeypatch.setattr(paged, "_workspace", lambda nbytes, device: (nbytes, device.index))
    q = SimpleNamespace(device=SimpleNamespace(index=1), dtype=paged.torch.bfloat16, shape=(1, 2, 64))
    assert paged.paged_tree_attention_workspace(q, SimpleNamespace(c=None), 1, 1) == (16, 1) and now == [0]
