"""Chunk attention on the GPU where a page's scale, or what a page outside a row's sight holds, decides: values are code x scale, and
nothing but the rows that a token sees counts.  Bounds as in test_gpu_paged_chunk.py unless a test derives its own."""
import numpy as np
import pytest
import torch

from test_gpu_paged_chunk import KINDS, Chunk

pytestmark = pytest.mark.gpu


ZERO_SCALES = [  # page, Hq, Hkv, D, lengths, window, pages of scale 0 (a request's i-th of m)
    (16, 4, 2, 128, [(300, 140), (0, 130), (700, 1)], 0, lambda i, m: i < m // 2),
    (128, 4, 2, 64, [(300, 140), (0, 130), (700, 1)], 0, lambda i, m: i < m // 2),
    (32, 4, 2, 128, [(300, 140), (0, 130), (700, 1)], 0, lambda i, m: i >= m // 2),
    (64, 4, 2, 128, [(300, 140), (0, 130), (700, 1)], 0, lambda i, m: True),
    # a unit in many CTAs' ranges: parts that begin in, or lie wholly in, zeros
    (64, 32, 4, 128, [(6000, 40)], 0, lambda i, m: i % 10 < 7),
    (128, 32, 4, 64, [(6000, 40)], 0, lambda i, m: 10 <= i < 40),
    # single tokens alone
    (16, 8, 2, 128, [(700, 1), (1500, 1), (40, 1), (5000, 1)], 0, lambda i, m: i < 2 * m // 3),
    (128, 48, 1, 64, [(700, 1), (1500, 1), (40, 1), (5000, 1)], 0, lambda i, m: i % 3 < 2),
    # the window begins in zeros
    (16, 4, 2, 128, [(1000, 200), (900, 3), (1200, 1)], 700, lambda i, m: i < 3 * m // 4),
    (128, 6, 2, 64, [(1000, 200), (900, 3), (1200, 1)], 300, lambda i, m: i < m - 1),
]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("case", ZERO_SCALES, ids=lambda c: "-".join(str(x) for x in c[:4]) + "-w%d" % c[5])
def test_codes_under_a_scale_of_zero_are_zero(tsv, kind, case):
    """Pages whose V scale is 0 and whose codes are not: they weigh, and add nothing.  Of the other KV heads the scale stays."""
    page, Hq, Hkv, D, lens, window, zero = case
    b = Chunk(tsv, np.random.default_rng(page + D), lens, Hq, Hkv, D, page, dtype=kind[1])
    for i, (p, n) in enumerate(lens):
        m = -(-(p + n) // page)
        ids = torch.tensor([b.table[i][x] for x in range(m) if zero(x, m)], device="cuda", dtype=torch.int64)
        assert (b.cache.v.view(torch.uint8)[ids, :, 0] & 0x7F != 0).any()
        b.cache.v_scale[ids, 0] = 0.0
    out, st = b.run(tsv, flags=kind[2], window=window)
    b.check(out, st, kind[2], window=window)
    assert Hkv == 1 or not (out[:, Hq // Hkv:] == 0).all()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("case", [(16, 4, 2, 128, [(1000, 200), (900, 3), (1205, 1), (0, 150)], 100),
                                  (16, 32, 4, 64, [(6000, 40), (3333, 1)], 3000), (32, 6, 1, 128, [(411, 1), (500, 60)], 77)],
                         ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_scales_in_front_of_a_window_do_not_count(tsv, kind, case):
    """Pages in front of every row's window may have any scales: no bit of a result changes, with V values 2^100 times as large
    there."""
    page, Hq, Hkv, D, lens, window = case
    b = Chunk(tsv, np.random.default_rng(page + Hq), lens, Hq, Hkv, D, page, dtype=kind[1])
    want, st = b.run(tsv, flags=kind[2], window=window)
    b.check(want, st, kind[2], window=window)
    for i, (p, n) in enumerate(lens):
        front = max(0, p - window + 1) // page  # pages that no new row sees anything of
        ids = torch.from_numpy(b.table[i][:front].astype(np.int64)).cuda()
        b.cache.v_scale[ids] *= 2.0 ** 100
        b.cache.k_scale[ids] *= 2.0 ** 100
    out, st = b.run(tsv, flags=kind[2], window=window)
    assert (st == 0).all() and torch.equal(out, want)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("case", [(16, 4, 2, 128, [(1000, 200), (900, 3), (1205, 1), (0, 150), (333, 0)], 100),
                                  (16, 32, 4, 64, [(6000, 40), (3333, 1), (5, 0)], 3000), (128, 6, 1, 128, [(1411, 1), (500, 60)], 77)],
                         ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_pages_in_front_of_a_window_may_be_given_away(tsv, kind, case):
    """Entries of pages that no new row sees: out of range on either side, or other requests' pages of NaN codes under large
    scales.  The request stays valid and no bit changes; an entry of the first page that a row sees has to be right."""
    page, Hq, Hkv, D, lens, window = case
    b = Chunk(tsv, np.random.default_rng(page + Hq), lens, Hq, Hkv, D, page, dtype=kind[1])
    want, st = b.run(tsv, flags=kind[2], window=window)
    b.check(want, st, kind[2], window=window)
    unused = sorted(set(range(b.cache.num_pages)) - set(b.table[b.table >= 0].tolist()))
    b.cache.k.view(torch.uint8)[unused] = 0x7F
    b.cache.v.view(torch.uint8)[unused] = 0xFF
    b.cache.k_scale[unused] = b.cache.v_scale[unused] = 2.0 ** 100
    fronts = [max(0, p - window + 1) // page if n else -(-p // page) for p, n in lens]
    table = b.table.copy()
    for fill in (-1, b.cache.num_pages, 2 ** 31 - 1, unused[0]):
        for i, front in enumerate(fronts):
            b.table[i][:front] = fill
        out, st = b.run(tsv, flags=kind[2], window=window)
        assert st.tolist() == [0] * len(lens) and torch.equal(out, want)
    for i, front in enumerate(fronts):
        b.table = table.copy()
        b.table[i][front] = -1
        out, st = b.run(tsv, flags=kind[2], window=window)
        assert st.tolist() == [int(x == i and lens[i][1] > 0) for x in range(len(lens))]
        keep = torch.ones(len(out), dtype=torch.bool, device="cuda")
        keep[int(b.offs[i]):int(b.offs[i + 1])] = False
        assert torch.equal(out[keep], want[keep])
    # without a window every page counts
    b.table = table.copy()
    b.table[0][0] = -1
    _, st = b.run(tsv, flags=kind[2])
    assert st.tolist() == [1] + [0] * (len(lens) - 1)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_requests_without_new_rows_need_no_pages(tsv, kind):
    b = Chunk(tsv, np.random.default_rng(3), [(300, 20), (500, 0), (40, 1), (0, 0)], 4, 2, 64, 16, dtype=kind[1])
    b.table[1] = -1
    for kw in (dict(), dict(window=50)):
        out, st = b.run(tsv, flags=kind[2], **kw)
        b.check(out, st, kind[2], **kw)
    b.offs, b.q = np.array([0, 1, 1, 2, 2]), b.q[:2].contiguous()  # single tokens
    b.lens = [(300, 1), (500, 0), (40, 1), (0, 0)]
    out, st = b.run(tsv, flags=kind[2], max_rows=1)
    b.check(out, st, kind[2])
