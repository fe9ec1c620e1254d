"""Page lists on the GPU: how calls treat what the caller passes."""
import numpy as np
import pytest

import _pages_ref as P
from test_gpu_paged import i32
from test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


def test_compaction_leaves_the_callers_dict_alone(tsv):
    """Results without a status of their own: the returned dict has one, the passed one is as it was."""
    p = Pool(tsv, np.random.default_rng(1), 300, [20, 7, 30], 40)
    first = tsv.pages_compact(p.pool, [p.d_table], [p.d_pages])
    want = {k: v.clone() for k, v in first.items() if k not in ("tables", "status")}
    out = {k: v for k, v in first.items() if k != "status"}
    names = set(out)
    got = tsv.pages_compact(p.pool, [p.d_table], [p.d_pages], out=out)
    assert set(out) == names and got["status"].tolist() == [0]
    for k, v in want.items():
        assert got[k] is out[k]
        m = int(got["moved"]) if k.startswith("move_") else None  # (entries behind the moves are not written)
        assert (got[k][:m] == v[:m]).all()


def test_sources_and_lists_may_take_turns_in_one_table(tsv):
    """A table whose even rows are the sources of its odd rows, and one whose columns are split between them: as from two tables."""
    rng = np.random.default_rng(2)
    p = Pool(tsv, rng, 500, [20, 0, 33, 0, 7, 0, 40, 0], 48)
    table, pages = p.table, p.pages
    even, odd = [0, 2, 4, 6], [1, 3, 5, 7]
    source, rows = [2, 0, -1, 3], [7, 315, 5, 640]
    first, second = [table[b] for b in even], [table[b] for b in odd]
    held, to = p.d_pages[0::2].contiguous(), p.d_pages[1::2].contiguous()
    r = tsv.pages_fork(p.pool, p.d_table[0::2], held, i32(source), i32(rows), p.d_table[1::2], to, 16)
    child = [pages[b] for b in odd]
    want = P.fork(p.plain, first, [pages[b] for b in even], source, rows, second, child, 16)
    assert [r[k].tolist() for k in ("copy_src", "copy_dst", "status")] == [list(w) for w in want]
    for b, row in zip(odd, second):
        table[b] = row
    assert p.d_table.tolist() == table and to.tolist() == child and p.pool.refs.tolist() == p.plain.refs
    # columns: lists of 24 entries beside sources of 24
    q = Pool(tsv, rng, 500, [20, 24, 3], 48)
    to = i32([0, 0, 0])
    r = tsv.pages_fork(q.pool, q.d_table[:, :24], q.d_pages, i32([1, 2, 0]), i32([300, 48, 160]), q.d_table[:, 24:], to, 16)
    left, right, child = [t[:24] for t in q.table], [t[24:] for t in q.table], [0, 0, 0]
    want = P.fork(q.plain, left, q.pages, [1, 2, 0], [300, 48, 160], right, child, 16)
    assert [r[k].tolist() for k in ("copy_src", "copy_dst", "status")] == [list(w) for w in want]
    assert q.d_table.tolist() == [a + b for a, b in zip(left, right)] and to.tolist() == child
    with pytest.raises(tsv.TSVError):
        tsv.pages_fork(q.pool, q.d_table[:, :25], q.d_pages, i32([1, 2, 0]), i32([300, 48, 160]), q.d_table[:, 24:], to, 16)
