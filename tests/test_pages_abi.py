"""include/tsv_pages.h and the chunk attention of include/tsv_paged.h: exports, binding, host-side refusals (no device needed)."""
import ctypes
import math
import os
import re
import subprocess

import pytest

from test_paged_abi import H, P, _cache, _table, paged  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tsv_pages.h")


@pytest.fixture(scope="module")
def pages(paged):  # noqa: F811
    import tree_speculative_verification_attention_gb300 as tsv
    return tsv.pages


def test_exports_binding_and_constants(pages):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^tsv_status\s+(tsv_[a-z_]+)\s*\(", text, re.M))
    assert names == set(pages.PAGES_EXPORTED)
    for n in names:
        assert hasattr(pages._lib, n) and callable(getattr(pages, n))
    assert "#define TSV_PAGES_MAX_LISTS %d\n" % pages.TSV_PAGES_MAX_LISTS in text
    assert b"pages" in pages._lib.tsv_status_string(7)


def test_header_is_plain_c_and_structs_match_the_binding(pages, tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tsv_pages.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu %zu", sizeof(tsv_page_pool), offsetof(tsv_page_pool, num_pages), sizeof(tsv_page_lists), '
                   'offsetof(tsv_page_lists, out_d), offsetof(tsv_page_lists, out_stride), offsetof(tsv_page_lists, B));\nreturn 0; }\n')
    exe = tmp_path / "t"
    cc = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I" + os.path.join(ROOT, "include"),
                         str(src), "-o", str(exe)], capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    A, L = pages.CPagePool, pages.CPageLists
    assert got == [ctypes.sizeof(A), A.num_pages.offset, ctypes.sizeof(L), L.out_d.offset, L.out_stride.offset, L.B.offset]


# A block of zeros stands for a handle and made-up addresses for buffers: a refused call touches neither.


def _lists(pages, **kw):
    f = dict(table=pages.CPageTable(ids_d=P, stride=4, pages=4), pages_d=P, out_d=P + 4096, out_stride=4, B=2)
    f.update(kw)
    return pages.CPageLists(**f)


def _call(paged, name, **kw):  # noqa: F811
    import tree_speculative_verification_attention_gb300 as tsv
    pages = tsv.pages
    pool = kw.pop("pool", pages.CPagePool(refs_d=P, num_pages=64))
    table, other = kw.pop("table", _table(paged)), kw.pop("other", _table(paged, ids_d=P + 4096))
    cache, lists = kw.pop("cache", _cache(paged)), kw.pop("lists", _lists(pages))
    orders = {
        "tsv_pages_resize": dict(h=H, pool=pool, table=table, held=P, rows=P, B=2, page=16, status=P, stream=None),
        "tsv_pages_fork": dict(h=H, pool=pool, table=table, held=P, F=2, source=P, rows=P, other=other, to=P, B=2, page=16, src=P,
                               dst=P + 64, status=P, stream=None),
        "tsv_pages_compact": dict(h=H, pool=pool, refs=P, lists=lists, n=1, new=P + 1024, src=P, dst=P + 64, moved=P, status=P, stream=None),
        "tsv_pages_copy": dict(h=H, cache=cache, src=P, dst=P, n=5, count=None, status=P, stream=None),
        "tsv_paged_chunk_attention": dict(h=H, dtype=1, q=P, qn=256, qh=64, cache=cache, table=table, start=P, offs=P, out=P, B=2, N=5,
                                          max_rows=4, Hq=4, window=0, scale=0.0, ws=P, wsb=1 << 40, status=P, flags=0, stream=None),
    }
    args = orders[name]
    for k in kw:
        assert k in args, k
    args.update(kw)
    return getattr(paged._lib, name)(*[paged._at(x) if isinstance(x, ctypes.Structure) else x for x in args.values()])


BAD = {
    "tsv_pages_resize": [dict(h=None), dict(B=0), dict(B=129), dict(page=0), dict(held=None), dict(rows=None), dict(status=None)],
    "tsv_pages_fork": [dict(h=None), dict(B=0), dict(B=129), dict(F=0), dict(F=65537), dict(page=0), dict(held=None), dict(source=None),
                       dict(rows=None), dict(to=None), dict(src=None), dict(dst=None), dict(dst=P), dict(status=None)],
    "tsv_pages_compact": [dict(h=None), dict(n=-1), dict(n=9), dict(refs=None), dict(new=None), dict(new=P), dict(src=None),
                          dict(dst=None), dict(dst=P), dict(moved=None), dict(status=None)],
    "tsv_pages_copy": [dict(h=None), dict(n=-1), dict(src=None), dict(dst=None), dict(status=None)],
    "tsv_paged_chunk_attention": [dict(h=None), dict(dtype=-1), dict(flags=2), dict(B=0), dict(B=129), dict(max_rows=0), dict(Hq=0),
                                  dict(Hq=3), dict(start=None), dict(offs=None), dict(status=None), dict(N=-1), dict(window=-1),
                                  dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(q=None), dict(out=None),
                                  dict(out=P + 8), dict(q=P + 2), dict(qn=4), dict(qh=2)],
}


@pytest.mark.parametrize("name", sorted(BAD))
def test_bad_arguments_are_refused(paged, name):  # noqa: F811
    for kw in BAD[name]:
        assert _call(paged, name, **kw) == 1, (name, kw)


@pytest.mark.parametrize("name", ["tsv_pages_resize", "tsv_pages_fork", "tsv_pages_compact"])
def test_bad_pools_and_lists_are_refused(paged, pages, name):  # noqa: F811
    pool = pages.CPagePool
    for p in (None, pool(refs_d=None, num_pages=64), pool(refs_d=P + 4, num_pages=64), pool(refs_d=P, num_pages=0)):
        assert _call(paged, name, pool=p) == 1
    assert _call(paged, name, pool=pool(refs_d=P, num_pages=(1 << 27) + 1)) == 3
    if name == "tsv_pages_compact":
        wide = pages.CPageTable(ids_d=P, stride=4, pages=5)
        for kw in (dict(B=0), dict(pages_d=None), dict(out_d=None), dict(out_stride=3), dict(out_d=P, out_stride=8), dict(table=wide)):
            assert _call(paged, name, lists=_lists(pages, **kw)) == 1, kw
        assert _call(paged, name, lists=None) == 1
        big = pages.CPageTable(ids_d=P, stride=1 << 30, pages=1 << 30)
        assert _call(paged, name, lists=_lists(pages, table=big, out_stride=1 << 30, B=1 << 20)) == 3
        return
    for kw in (dict(ids_d=None), dict(pages=0), dict(stride=3), dict(ids_d=P + 2)):
        assert _call(paged, name, table=_table(paged, **kw)) == 1, kw
        if name == "tsv_pages_fork":
            assert _call(paged, name, other=_table(paged, **kw)) == 1, kw
    assert _call(paged, name, table=_table(paged, pages=(1 << 30) + 1, stride=1 << 31)) == 3


def test_forked_lists_do_not_overlap_their_sources(paged):  # noqa: F811
    for ids in (P, P + 16, P - 16, P + 28):  # two rows of four entries each
        assert _call(paged, "tsv_pages_fork", other=_table(paged, ids_d=ids)) == 1


@pytest.mark.parametrize("name", ["tsv_pages_copy", "tsv_paged_chunk_attention"])
def test_bad_caches_are_refused(paged, name):  # noqa: F811
    for kw in (dict(k_d=None), dict(v_d=P + 8), dict(k_scale_d=None), dict(v_scale_d=P + 2), dict(num_pages=0), dict(Hkv=0),
               dict(stride_row=0), dict(stride_row=72), dict(stride_head=-64), dict(stride_page=8)):
        assert _call(paged, name, cache=_cache(paged, **kw)) == 1, kw
    for kw in (dict(D=96), dict(page_size=8), dict(page_size=48), dict(num_pages=1 << 28)):
        assert _call(paged, name, cache=_cache(paged, **kw)) == 3, kw
    assert _call(paged, name, cache=None) == 1
    if name == "tsv_paged_chunk_attention":
        for kw in (dict(ids_d=None), dict(pages=0), dict(stride=3)):
            assert _call(paged, name, table=_table(paged, **kw)) == 1, kw
        assert _call(paged, name, N=1 << 30, B=1, Hq=2) == 3
    else:  # a page of more than 2^33 bytes
        assert _call(paged, name, cache=_cache(paged, Hkv=(1 << 23) + 1)) == 3


def test_chunk_workspace_size_refusals(paged):  # noqa: F811
    n = ctypes.c_size_t(7)
    f = lambda h, dt, c, *a: paged._lib.tsv_paged_chunk_attention_workspace_size(h, dt, paged._at(c), *a)  # noqa: E731
    c = _cache(paged)
    for bad in ((None, 1, c, 1, 1, 1, 4, 0, ctypes.byref(n)), (H, 1, c, 1, 1, 1, 4, 0, None), (H, 1, c, 1, 1, 1, 3, 0, ctypes.byref(n)),
                (H, 1, c, 1, -1, 1, 4, 0, ctypes.byref(n)), (H, 1, c, 1, 1, 0, 4, 0, ctypes.byref(n)),
                (H, 1, c, 0, 1, 1, 4, 0, ctypes.byref(n))):
        assert f(*bad) == 1
    assert f(H, 1, _cache(paged, D=32), 1, 1, 1, 4, 0, ctypes.byref(n)) == 3
    assert n.value == 7


def test_good_arguments_reach_the_device(paged):  # noqa: F811
    """The arguments that the refusals above start from are accepted: what stops them here is that there is no device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present: the made-up addresses must not reach it")
    for name in BAD:
        assert _call(paged, name) == 4, name
