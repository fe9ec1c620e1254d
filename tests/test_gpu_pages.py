"""Page lists on the GPU against the plain forms of tests/_pages_ref.py: whole numbers and codes, equal to the last bit."""
import numpy as np
import pytest
import torch

import _pages_ref as P
from test_gpu_paged import dev, i32, make_cache

pytestmark = pytest.mark.gpu


def lists_of(t):
    return [list(map(int, row)) for row in t]


class Pool:
    """Random lists over a pool, on the device and as plain lists."""

    def __init__(self, tsv, rng, num_pages, held, width, shared=0.0, other=0.0, counts=None):
        ids = rng.permutation(num_pages)
        table = np.full((len(held), width), -7, dtype=np.int32)
        refs = np.zeros(num_pages, dtype=np.int32)
        at = 0
        for b, n in enumerate(held):
            share = min(int(held[b - 1] * shared), n) if b else 0
            table[b, :share] = table[b - 1, :share]
            table[b, share:n] = ids[at:at + n - share]
            at += n - share
            np.add.at(refs, table[b, :n], 1)
        refs[ids[at:at + int((num_pages - at) * other)]] = 3  # held by lists that no call sees
        if counts is not None:
            refs = counts(refs)
        self.plain, self.table, self.pages = P.Pool(refs), lists_of(table), list(map(int, held))
        self.d_table, self.d_pages, self.pool = dev(table), i32(held), tsv.PagePool(dev(refs))

    def same(self):
        assert self.pool.refs.tolist() == self.plain.refs
        assert self.d_pages.tolist() == self.pages
        assert self.d_table.tolist() == self.table

    def resize(self, tsv, rows, page, **kw):
        st = tsv.pages_resize(self.pool, self.d_table, self.d_pages, i32(rows), page, **kw)
        want = P.resize(self.plain, self.table, self.pages, rows, page)
        assert st.tolist() == want
        self.same()
        return want


SIZES = [  # pages of the pool, lists, most entries
    (1, 1, 1), (7, 2, 3), (129, 3, 40), (4096, 16, 200), (4097, 128, 30), (20000, 33, 500), (70001, 128, 400), (300000, 20, 9000),
]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_resize(tsv, size):
    pages, B, W = size
    rng = np.random.default_rng(pages)
    p = Pool(tsv, rng, pages, np.minimum(rng.integers(0, W + 1, size=B), pages // B), W, other=0.3)
    for page in (16, 1, 128, 5):
        for most in (W, W // 2, W // 8):
            p.resize(tsv, [int(x) for x in rng.integers(0, most * page + 1, size=B)], page)
        p.resize(tsv, [n * page for n in p.pages], page)  # nothing changes
    st = p.resize(tsv, [0] * B, 16)
    assert st == [0] * B and p.pages == [0] * B


def test_resize_without_enough_pages(tsv):
    """The requests before the first that does not fit get theirs, those behind it that need none are fine."""
    rng = np.random.default_rng(1)
    p = Pool(tsv, rng, 5000, [100] * 30, 400, other=0.5)
    seen = set()
    for k in range(6):
        seen |= set(p.resize(tsv, [int(x) for x in rng.choice([50 * 16, 100 * 16, 200 * 16, 400 * 16], size=30)], 16))
    assert seen == {0, 7}
    q = Pool(tsv, rng, 64, [0] * 3, 64)
    assert q.resize(tsv, [16 * 64, 1, 0], 16) == [0, 7, 0]  # all of the pool
    # needs whose sum passes 32 bits: 128 requests of 2^26 pages each
    wide = torch.full((128, 1), -7, dtype=torch.int32, device="cuda").expand(128, 1 << 26)
    held = i32([0] * 128)
    with pytest.raises(ValueError):
        tsv.pages_resize(q.pool, wide, held, i32([1 << 26] * 128), 1)
    big = torch.empty(1 << 27, dtype=torch.int32, device="cuda").as_strided((128, 1 << 20), (1 << 20, 1))
    big.fill_(-7)
    r = tsv.PagePool(torch.zeros(1000, dtype=torch.int32, device="cuda"))
    st = tsv.pages_resize(r, big, held, i32([1 << 20] * 127 + [5]), 1)
    assert st.tolist() == [7] * 128 and (held == 0).all() and (r.refs == 0).all() and (big == -7).all()
    st = tsv.pages_resize(r, big, held, i32([3, 900] + [1 << 20] * 125 + [5]), 1)
    assert st.tolist() == [0, 0] + [7] * 126 and int(r.refs.sum()) == 903


def test_resize_rejects_requests_one_by_one(tsv):
    rng = np.random.default_rng(2)
    p = Pool(tsv, rng, 600, [10, 10, 10, 10, 10, 10, 4], 12, shared=0.5)
    p.table[0][8], p.table[1][9], p.pages[2], p.pages[3] = 600, -1, 13, -1
    p.d_table, p.d_pages = i32(p.table), i32(p.pages)
    # out of range, out of range, too many held, fewer than none, more wanted than fit, negative rows, fine
    assert p.resize(tsv, [16, 16, 16, 16, 16 * 12 + 1, -5, 100], 16) == [1, 1, 1, 1, 1, 1, 0]
    # a page that is not held; rows that end in a page that the list before holds too
    p = Pool(tsv, rng, 600, [10, 10], 12, shared=0.5)
    free = p.plain.refs.index(0)
    p.table[0][9] = free
    p.d_table = i32(p.table)
    assert p.resize(tsv, [16, 16 * 5 - 3], 16) == [1, 1]
    assert p.resize(tsv, [16 * 9, 16 * 5], 16) == [1, 0]
    # pages listed more often than they count: every count stays within 0 and what it was
    q = Pool(tsv, rng, 100, [8, 8], 8)
    q.d_table[1] = q.d_table[0]
    st = tsv.pages_resize(q.pool, q.d_table, q.d_pages, i32([0, 0]), 16)
    assert 1 in st.tolist() and q.pool.refs[q.d_table[0].long()].eq(0).all() and (q.pool.refs >= 0).all()


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("page", [16, 7])
def test_fork(tsv, size, page):
    pages, B, W = size
    rng = np.random.default_rng(pages + page)
    F = max(1, B // 4)
    held = np.minimum(rng.integers(0, W + 1, size=F + B), pages // (2 * (F + B)))
    p = Pool(tsv, rng, pages, held, W, shared=0.3, other=0.2)
    for step in range(4):
        src = [int(x) for x in rng.integers(-1, F, size=B)]
        rows = [int(rng.integers(0, p.pages[s] * page + 1)) if s >= 0 else -3 for s in src]
        old = p.d_table.clone()
        out = tsv.pages_fork(p.pool, p.d_table[:F], p.d_pages[:F], i32(src), i32(rows), p.d_table[F:], p.d_pages[F:], page)
        child, has = p.table[F:], p.pages[F:]
        want = P.fork(p.plain, p.table[:F], p.pages[:F], src, rows, child, has, page)
        p.table[F:], p.pages[F:] = child, has
        assert [out[x].tolist() for x in ("copy_src", "copy_dst", "status")] == list(want)
        p.same()
        assert torch.equal(old[:F], p.d_table[:F])


def test_fork_without_enough_pages_and_bad_lists(tsv):
    rng = np.random.default_rng(4)
    p = Pool(tsv, rng, 40, [10, 8, 1, 1, 1, 1, 1, 1], 12, other=1.0)
    page = 16

    def call(src, rows):
        out = tsv.pages_fork(p.pool, p.d_table[:2], p.d_pages[:2], i32(src), i32(rows), p.d_table[2:], p.d_pages[2:], page)
        child, has = p.table[2:], p.pages[2:]
        want = P.fork(p.plain, p.table[:2], p.pages[:2], src, rows, child, has, page)
        p.table[2:], p.pages[2:] = child, has
        assert [out[x].tolist() for x in ("copy_src", "copy_dst", "status")] == list(want)
        p.same()
        return want[2]

    # four lists give their page back, five want one of their own and one shares whole pages
    assert call([0, 1, 0, -1, 0, 1], [150, 100, 32, 5, 33, 1]) == [0, 0, 0, 0, 0, 0]
    # five pages come back and one was left: five are wanted, and then six of them when one is kept by somebody else
    assert call([0, 1, 0, 1, 0, 1], [31, 33, 47, 48, 65, 17]) == [0, 0, 0, 0, 0, 0]
    kept = p.plain.free()[0]
    p.plain.refs[kept] = 1
    p.pool.refs[kept] = 1
    assert call([0, 1, 0, 1, 0, 1], [31, 33, 47, 49, 65, 17]) == [0, 0, 0, 0, 0, 7]
    # sources and rows that do not fit
    assert call([2, -2, 0, 1, 0, -1], [1, 1, 161, -1, 160, 0]) == [1, 1, 1, 1, 0, 0]
    p.table[0][3], p.table[4][0], p.pages[5] = 40, -1, 13
    p.pages[4] = max(1, p.pages[4])
    p.d_table, p.d_pages = i32(p.table), i32(p.pages)
    assert call([0, 0, 1, 1, 1, 1], [64, 48, 16, 16, 128, 0]) == [1, 0, 1, 1, 0, 0]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(tsv, size, in_place):
    pages, B, W = size
    rng = np.random.default_rng(pages + 1)
    for fill, other in ((2, 0.3), (1, 0.0), (1, 1.0), (100, 0.0)):
        held = np.minimum(rng.integers(0, W + 1, size=B), pages // (B * fill))
        p = Pool(tsv, rng, pages, held, W, shared=0.2, other=other)
        second = rng.integers(0, 3, size=300)
        more = i32([[p.table[b % B][i] if i < min(second[b], held[b % B]) else -9 for i in range(3)] for b in range(300)])
        n2 = i32(np.minimum(second, held[np.arange(300) % B]))
        want = P.compact(p.plain, [p.table, lists_of(more.tolist())], [p.pages, n2.tolist()])
        tables = [p.d_table, more]
        before = [t.clone() for t in tables]
        out = tsv.pages_compact(p.pool, tables, [p.d_pages, n2], in_place=in_place)
        refs, new_id, src, dst, lists, st = want
        m = int(out["moved"])
        assert m == len(src) and out["move_src"][:m].tolist() == src and out["move_dst"][:m].tolist() == dst
        assert out["refs"].tolist() == refs and out["new_id"].tolist() == new_id and out["status"].tolist() == st == [0, 0]
        assert (out["refs"] is p.pool.refs) == in_place
        for got, line, was in zip(out["tables"], lists, before):
            mask = torch.tensor([[x is not None for x in row] for row in line], device="cuda")
            w = i32([[-1 if x is None else x for x in row] for row in line])
            assert torch.equal(got[mask], w[mask])
            if in_place:
                assert torch.equal(got[~mask], was[~mask])


def test_compact_reports_bad_lists_and_takes_none(tsv):
    rng = np.random.default_rng(6)
    p = Pool(tsv, rng, 300, [20, 20, 20], 30)
    out = tsv.pages_compact(p.pool, [], [])
    refs, new_id, src, dst, _, _ = P.compact(p.plain, [], [])
    assert out["refs"].tolist() == refs and out["new_id"].tolist() == new_id and int(out["moved"]) == len(src)
    free = p.plain.refs.index(0)
    for bad in (dict(entry=300), dict(entry=-1), dict(entry=free), dict(count=31), dict(count=-1)):
        table, pages = p.d_table.clone(), p.d_pages.clone()
        if "entry" in bad:
            table[1, 5] = bad["entry"]
        else:
            pages[1] = bad["count"]
        out = tsv.pages_compact(p.pool, [p.d_table, table], [p.d_pages, pages])
        want = P.compact(p.plain, [p.table, lists_of(table.tolist())], [p.pages, pages.tolist()])
        assert out["status"].tolist() == want[5] == [0, 1]
        for row, line in zip(out["tables"][1].tolist(), want[4][1]):
            assert all(x == y for x, y in zip(row, line) if y is not None)


COPY = [  # pages, page, Hkv, D, layout
    (9, 16, 8, 128, "head"), (40, 64, 3, 64, "token"), (12, 128, 1, 128, "head"), (30, 16, 5, 64, "fused"), (300, 32, 2, 128, "fused"),
    (20, 64, 2, 64, "holes"), (5, 128, 32, 128, "head"),
]


def cache_of(tsv, rng, pages, page, Hkv, D, layout):
    shape = {"head": (2, pages, Hkv, page, D), "token": (2, pages, page, Hkv, D), "fused": (pages, page, 2, Hkv, D),
             "holes": (2, pages + 1, Hkv + 1, page + 2, D + 16)}[layout]
    x = dev(rng.integers(0, 256, size=shape, dtype=np.uint8))
    if layout == "head":
        k, v = x[0].transpose(1, 2), x[1].transpose(1, 2)
    elif layout == "token":
        k, v = x[0], x[1]
    elif layout == "fused":
        k, v = x[:, :, 0], x[:, :, 1]
    else:
        k, v = (x[i, :pages, 1:, 1:-1, :D].transpose(1, 2) for i in range(2))
    s = [dev(rng.random((pages, Hkv)), torch.float32) for _ in range(2)]
    return tsv.PagedCache(k, v, *s), x


@pytest.mark.parametrize("case", COPY, ids=lambda c: "-".join(map(str, c)))
def test_copy(tsv, case):
    pages, page, Hkv, D, layout = case
    rng = np.random.default_rng(pages)
    c, x = cache_of(tsv, rng, *case)
    ids = rng.permutation(pages)
    n = pages // 2
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    src[n // 3:n // 3 + 1] = -1
    if n > 2:
        dst[n - 1] = -1
    whole = x.clone()
    want = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            for t in want:
                t[b] = t[a].clone()
    st = tsv.pages_copy(c, i32(src), i32(dst))
    assert st.tolist() == [0]
    for t, w in zip((c.k, c.v, c.k_scale, c.v_scale), want):
        assert torch.equal(t, w)
    # what lies outside of the cache's elements stays
    back = x.clone()
    if layout == "holes":
        for i in range(2):
            back[i, :pages, 1:, 1:-1, :D] = whole[i, :pages, 1:, 1:-1, :D]
        assert torch.equal(back, whole)


def test_copy_counts_and_bad_ids(tsv):
    rng = np.random.default_rng(7)
    c, _ = cache_of(tsv, rng, 50, 16, 2, 64, "head")
    src, dst = i32(range(20)), i32(range(20, 40))
    for count, copied in ((0, 0), (-4, 0), (7, 7), (20, 20), (1 << 30, 20)):
        before = c.k.clone()
        assert tsv.pages_copy(c, src, dst, count=i32([count])).tolist() == [0]
        assert torch.equal(c.k[20:20 + copied], before[:copied]) and torch.equal(c.k[20 + copied:], before[20 + copied:])
        c.k[20:] = dev(rng.integers(0, 256, size=(30, 16, 2, 64), dtype=np.uint8))
    before = c.k.clone()
    for bad in (50, -2, 1 << 30):
        for which in (src, dst):
            was = int(which[3])
            which[3] = bad
            assert tsv.pages_copy(c, src, dst).tolist() == [1]
            assert tsv.pages_copy(c, src, dst, count=i32([3])).tolist() == [0]  # (behind the count: not looked at)
            assert torch.equal(c.k[24:40], before[4:20]) and torch.equal(c.k[23], before[23])
            which[3] = was
    assert tsv.pages_copy(c, i32([]), i32([])).tolist() == [0]


def test_shapes_and_types_are_refused(tsv):
    rng = np.random.default_rng(8)
    p = Pool(tsv, rng, 100, [3, 3, 3], 5)
    c = make_cache(tsv, rng, 8, 16, 2, 64, True)
    t, n = p.d_table, p.d_pages
    for bad in (lambda: tsv.pages_resize(p.pool, t, n[:2], i32([1, 1, 1]), 16), lambda: tsv.pages_resize(p.pool, t, n, i32([1, 1]), 16),
                lambda: tsv.pages_resize(p.pool, t.long(), n, i32([1, 1, 1]), 16),
                lambda: tsv.pages_resize(p.pool, t[:, ::2], n, i32([1, 1, 1]), 16),
                lambda: tsv.pages_resize(p.pool, t, n.cpu(), i32([1, 1, 1]), 16),
                lambda: tsv.pages_fork(p.pool, t[:1], n, i32([0, 0]), i32([1, 1]), t[1:], n[1:], 16),
                lambda: tsv.pages_fork(p.pool, t[:1], n[:1], i32([0]), i32([1, 1]), t[1:], n[1:], 16),
                lambda: tsv.pages_compact(p.pool, [t], []), lambda: tsv.pages_compact(p.pool, [t] * 9, [n] * 9),
                lambda: tsv.pages_copy(c, i32([1]), i32([1, 2])), lambda: tsv.pages_copy(c, i32([1]), i32([2]).float()),
                lambda: tsv.PagePool(torch.zeros(4, 2, dtype=torch.int32, device="cuda")),
                lambda: tsv.PagePool(torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tsv.TSVError):  # a list is not a fork of itself
        tsv.pages_fork(p.pool, t[:2], n[:2], i32([0, 0]), i32([1, 1]), t[1:], n[1:], 16)
    with pytest.raises(tsv.TSVError):
        tsv.pages_resize(p.pool, t, n, i32([1, 1, 1]), 0)
    p.same()


def test_captured_calls_follow_the_lists(tsv):
    """A captured resize, fork, compaction and copy read lists and counts at the time of the replay; on a stream of its own."""
    rng = np.random.default_rng(9)
    p = Pool(tsv, rng, 9000, [30] * 8, 64, other=0.5)
    c = make_cache(tsv, rng, 9000, 16, 2, 64, True)
    rows, st = i32([0] * 8), i32([0] * 8)
    src, frows = i32([0] * 4), i32([0] * 4)
    out = dict(copy_src=i32([0] * 4), copy_dst=i32([0] * 4), status=i32([0] * 4))

    def step():
        tsv.pages_resize(p.pool, p.d_table, p.d_pages, rows, 16, status=st)
        tsv.pages_fork(p.pool, p.d_table[:4], p.d_pages[:4], src, frows, p.d_table[4:], p.d_pages[4:], 16, out=out)
        tsv.pages_copy(c, out["copy_src"], out["copy_dst"], status=cst)

    cst = i32([5])
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    saved = [t.clone() for t in (p.pool.refs, p.d_table, p.d_pages)]
    with torch.cuda.stream(s):
        step()  # (sets the kernels up)
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for t, was in zip((p.pool.refs, p.d_table, p.d_pages), saved):
        t.copy_(was)
    for k in range(5):
        r = [int(x) for x in rng.integers(1, 60, size=8) * 16]
        f, fr = [int(x) for x in rng.integers(0, 4, size=4)], [int(x) for x in rng.integers(1, 16, size=4)]
        rows.copy_(i32(r)), src.copy_(i32(f)), frows.copy_(i32(fr))
        codes = c.k.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert st.tolist() == P.resize(p.plain, p.table, p.pages, r, 16)
        child, has = p.table[4:], p.pages[4:]
        want = P.fork(p.plain, p.table[:4], p.pages[:4], f, fr, child, has, 16)
        p.table[4:], p.pages[4:] = child, has
        assert [out[x].tolist() for x in ("copy_src", "copy_dst", "status")] == list(want)
        p.same()
        assert cst.tolist() == [0] and torch.equal(c.k[out["copy_dst"].long()], codes[out["copy_src"].long()])


def test_lists_on_a_given_stream(tsv):
    """Calls go to the stream that they are given, behind what runs there already."""
    rng = np.random.default_rng(10)
    p = Pool(tsv, rng, 2000, [30] * 8, 64)
    s = torch.cuda.Stream()
    late = [int(x) for x in rng.integers(1, 60, size=8) * 16]
    rows, want = i32([0] * 8), i32(late)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)
        rows.copy_(want)
    st = tsv.pages_resize(p.pool, p.d_table, p.d_pages, rows, 16, stream=s)
    out = tsv.pages_compact(p.pool, [p.d_table], [p.d_pages], stream=s)
    s.synchronize()
    assert st.tolist() == P.resize(p.plain, p.table, p.pages, late, 16)
    p.same()
    refs, new_id = P.compact(p.plain, [], [])[:2]
    assert out["refs"].tolist() == refs and out["new_id"].tolist() == new_id
