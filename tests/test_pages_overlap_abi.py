"""tsv_pages_fork's check that lists and their sources lie apart (host side, no device needed)."""
import itertools

import pytest

from test_pages_abi import _call, pages  # noqa: F401
from test_paged_abi import P, _table, paged  # noqa: F401


def _reached(paged, first, second, F, B):  # noqa: F811
    """Whether the call is accepted: what stops it then is that there is no device."""
    return {1: False, 4: True}[_call(paged, "tsv_pages_fork", table=first, other=second, F=F, B=B)]


def _entries(t, rows):
    return {t.ids_d // 4 + b * t.stride + i for b in range(rows) for i in range(t.pages)}


def test_lists_that_take_turns_are_apart(paged):  # noqa: F811
    """Rows of one table in turn (sources the even ones, lists the odd ones), halves of its columns, and others: accepted exactly
    when no entry is in both."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present: the made-up addresses must not reach it")
    t = lambda at, stride, width: _table(paged, ids_d=P + 4 * at, stride=stride, pages=width)  # noqa: E731
    assert _reached(paged, t(0, 16, 8), t(8, 16, 8), 3, 3)      # in turn, whole rows
    assert _reached(paged, t(0, 16, 5), t(5, 16, 11), 9, 4)     # halves of columns
    assert not _reached(paged, t(0, 16, 6), t(5, 16, 11), 9, 4)
    assert _reached(paged, t(0, 1 << 40, 5), t(1 << 20, 1 << 40, 5), 65536, 128)
    assert not _reached(paged, t(0, 1 << 40, 5), t((1 << 41) - 4, 1 << 40, 5), 65536, 128)
    seen = set()
    for at, s1, s2, w1, w2, F, B in itertools.product((0, 1, 3, 8, 30, 61), (4, 7, 16), (4, 5, 16, 33), (1, 4), (1, 3, 4), (1, 2, 5), (1, 3)):
        for first, second in ((t(0, s1, w1), t(at, s2, w2)), (t(at, s1, w1), t(0, s2, w2))):
            apart = not (_entries(first, F) & _entries(second, B))
            assert _reached(paged, first, second, F, B) == apart, (at, s1, s2, w1, w2, F, B)
            seen.add(apart)
    assert seen == {True, False}
