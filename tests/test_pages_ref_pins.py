"""The plain forms of tests/_pages_ref.py by hand-worked cases and by what must hold of any."""
import numpy as np

import _paged_ref as R
import _pages_ref as P


def test_resize_by_hand():
    pool = P.Pool([0, 1, 0, 1, 1, 0, 0])
    table, pages = [[1, -1, -1], [3, 4, -1], [-1, -1, -1]], [1, 2, 0]
    assert P.resize(pool, table, pages, [40, 16, 17], 16) == [0, 0, 0]
    # request 1 gives page 4 back; request 0 takes 0 and 2, request 2 takes 4 and 5
    assert table == [[1, 0, 2], [3, 4, -1], [4, 5, -1]] and pages == [3, 1, 2]
    assert pool.refs == [1, 1, 1, 1, 1, 1, 0]
    # one page is left: request 1 wants two more, request 2 behind it one; request 0 wants none
    assert P.resize(pool, table, pages, [48, 33, 40], 16) == [0, 7, 7]
    assert pages == [3, 1, 2] and pool.refs[6] == 0
    assert P.resize(pool, table, pages, [-1, 49, 0], 16) == [1, 1, 0]
    assert pages == [3, 1, 0] and pool.refs == [1, 1, 1, 1, 0, 0, 0]


def test_a_list_does_not_shrink_into_a_shared_page():
    pool = P.Pool([2, 1])
    table, pages = [[0, 1]], [2]
    assert P.resize(pool, table, pages, [7], 8) == [1] and pages == [2]
    assert P.resize(pool, table, pages, [8], 8) == [0] and pages == [1] and pool.refs == [2, 0]


def test_fork_by_hand():
    pool = P.Pool([1, 1, 1, 2, 0, 0])
    parents, held = [[3, 0, 1]], [3]
    table, pages = [[2, -1, -1], [3, -1, -1], [-1, -1, -1]], [1, 1, 0]
    src, dst, st = P.fork(pool, parents, held, [0, 0, -1], [33, 32, 5], table, pages, 16)
    # page 2 comes back and is the lowest free one; both share 3 and 0
    assert (src, dst, st) == ([1, -1, -1], [2, -1, -1], [0, 0, 0])
    assert table[:2] == [[3, 0, 2], [3, 0, -1]] and pages == [3, 2, 0]
    assert pool.refs == [3, 1, 1, 3, 0, 0]
    assert P.fork(pool, parents, held, [0, 1, 0], [49, 1, 0], table, pages, 16)[2] == [1, 1, 0]


def test_counts_add_up_over_random_calls():
    rng = np.random.default_rng(0)
    pool, W, B, page = P.Pool([0] * 40), 8, 6, 4
    table, pages = [[-1] * W for _ in range(B)], [0] * B
    for step in range(300):
        if rng.random() < 0.5:
            P.resize(pool, table, pages, [int(x) for x in rng.integers(0, W * page + 1, size=B)], page)
        else:
            half = B // 2
            src = [int(x) for x in rng.integers(-1, half, size=half)]
            rows = [int(rng.integers(0, pages[s] * page + 1)) if s >= 0 else 0 for s in src]
            child, held = [list(t) for t in table[half:]], pages[half:]
            P.fork(pool, table[:half], pages[:half], src, rows, child, held, page)
            table[half:], pages[half:] = child, held
        count = np.zeros(40, dtype=int)
        for t, n in zip(table, pages):
            assert len(set(t[:n])) == n
            np.add.at(count, t[:n], 1)
        assert count.tolist() == pool.refs
        if step % 50 == 49:
            refs, new_id, src, dst, out, st = P.compact(pool, [table], [pages])
            live = sum(r > 0 for r in refs)
            assert all(r > 0 for r in refs[:live]) and not any(refs[live:]) and st == [0]
            assert sorted(new_id) == [-1] * (40 - live) + list(range(live))
            assert [new_id[s] for s in src] == dst and src == sorted(src) and dst == sorted(dst)
            pool = P.Pool(refs)
            table = [[x if x is not None else -1 for x in row] for row in out[0]]


def test_chunk_attention_is_the_tree_attention_of_a_chain():
    """Rows that lie in the prefix pages, against the same rows as a chain of tree rows behind a shorter prefix."""
    rng = np.random.default_rng(1)
    page, Hkv, D, Hq = 4, 2, 8, 6
    cache = R.Cache(rng.normal(size=(9, page, Hkv, D)), rng.normal(size=(9, page, Hkv, D)), np.ones((9, Hkv)), np.ones((9, Hkv)))
    q = rng.normal(size=(7, Hq, D))
    table = [[4, 2, 7, 1], [0, 3, -1, -1]]
    out, spread, size = P.chunk_attention(q, cache, table, [8, 4], [0, 3, 7])
    want, wspread, wsize = R.attention(q, cache, table, [8, 4], [0, 3, 7], tree_table=[[7, 1], [3, -1]])
    assert np.allclose(out, want) and np.allclose(spread, wspread) and np.allclose(size, wsize)
    # a window of one is the row's own value
    own, _, _ = P.chunk_attention(q, cache, table, [8, 4], [0, 3, 7], window=1)
    assert np.allclose(own[1], np.repeat(cache.v[7, 1], 3, axis=0))
    wide, _, _ = P.chunk_attention(q, cache, table, [8, 4], [0, 3, 7], window=100)
    assert np.allclose(wide, out)
