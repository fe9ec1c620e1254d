"""Plain forms of the page lists' operators and of the attention of a chunk, from their definitions in include/tsv_pages.h and
include/tsv_paged.h: one request, list and page at a time (lists and counts as Python integers, attention in 64 bits)."""
import math

import numpy as np

OK, INVALID, NO_PAGES = 0, 1, 7


def pages_of(rows, page):
    return -(-rows // page)


class Pool:
    def __init__(self, refs):
        self.refs = [int(r) for r in refs]

    def held(self, p):
        return 0 <= p < len(self.refs) and self.refs[p] > 0

    def free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]


def _serve(needs, free):
    """For each request whether it gets its pages, and the ids: in order, until the first that there are too few for."""
    out, at, over = [], 0, False
    for n in needs:
        over = over or (n > 0 and n > len(free) - at)
        if n > 0 and over:
            out.append(None)
            continue
        out.append(free[at:at + n])
        at += n
    return out


def resize(pool, table, pages, rows, page):
    """In place (table: lists of ids with the table's width); returns the status of each request."""
    status, want = [], []
    for b, r in enumerate(rows):
        w = pages_of(r, page) if r >= 0 else -1
        bad = r < 0 or not 0 <= pages[b] <= len(table[b]) or w > len(table[b])
        if not bad and w < pages[b]:
            bad = any(not pool.held(p) for p in table[b][w:pages[b]])
            if r % page:
                p = table[b][w - 1]
                bad = bad or not pool.held(p) or pool.refs[p] > 1
        status.append(INVALID if bad else OK)
        want.append(pages[b] if bad else w)
    for b, w in enumerate(want):
        for p in table[b][w:pages[b]] if status[b] == OK else []:
            pool.refs[p] -= 1
    got = _serve([max(0, w - n) if s == OK else 0 for w, n, s in zip(want, pages, status)], pool.free())
    for b, ids in enumerate(got):
        if ids is None:
            status[b] = NO_PAGES
            continue
        if status[b] != OK:
            continue
        for i, p in enumerate(ids):
            table[b][pages[b] + i] = p
            pool.refs[p] = 1
        pages[b] = want[b]
    return status


def fork(pool, source_table, source_pages, source, rows, table, pages, page):
    """In place; returns copy_src, copy_dst and the status of each list."""
    B = len(source)
    status, take = [OK] * B, [False] * B
    for b, (s, r) in enumerate(zip(source, rows)):
        if s == -1:
            continue
        w = pages_of(r, page) if r >= 0 else -1
        bad = not 0 <= s < len(source_table) or r < 0 or not 0 <= pages[b] <= len(table[b])
        bad = bad or not 0 <= source_pages[s] <= len(source_table[s]) or w > source_pages[s] or w > len(table[b])
        bad = bad or any(not pool.held(p) for p in table[b][:pages[b]] + source_table[s][:w])
        status[b], take[b] = INVALID if bad else OK, not bad
    for b in range(B):
        for p in table[b][:pages[b]] if take[b] else []:
            pool.refs[p] -= 1
    got = _serve([1 if take[b] and rows[b] % page else 0 for b in range(B)], pool.free())
    src, dst = [-1] * B, [-1] * B
    for b in range(B):
        if not take[b]:
            continue
        if got[b] is None:
            status[b], pages[b] = NO_PAGES, 0
            continue
        full = rows[b] // page
        for i in range(full):
            table[b][i] = source_table[source[b]][i]
            pool.refs[table[b][i]] += 1
        if got[b]:
            p = got[b][0]
            table[b][full], pool.refs[p] = p, 1
            src[b], dst[b] = source_table[source[b]][full], p
        pages[b] = pages_of(rows[b], page)
    return src, dst, status


def compact(pool, tables, counts):
    """Returns refs, new_id, move_src, move_dst, the tables (None: not written) and a status per table."""
    live = [p for p, r in enumerate(pool.refs) if r > 0]
    L = len(live)
    holes = iter([p for p in range(L) if pool.refs[p] <= 0])
    new_id, refs, src, dst = [-1] * len(pool.refs), [0] * len(pool.refs), [], []
    for p in live:
        new_id[p] = p if p < L else next(holes)
        if p >= L:
            src.append(p)
            dst.append(new_id[p])
        refs[new_id[p]] = pool.refs[p]
    out, status = [], []
    for table, n in zip(tables, counts):
        st, now = OK, []
        for row, m in zip(table, n):
            line = [None] * len(row)
            if 0 <= m <= len(row):
                for i, p in enumerate(row[:m]):
                    line[i] = new_id[p] if 0 <= p < len(new_id) else -1
                    if line[i] < 0:
                        st = INVALID
            else:
                st = INVALID
            now.append(line)
        out.append(now)
        status.append(st)
    return refs, new_id, src, dst, out, status


def chunk_attention(q, cache, table, start, row_offsets, window=0, scale=None):
    """Returns out [N, Hq, D], the same sums over |v|, and the largest scale * sum |q| |k| over the seen keys [N, Hq]."""
    N, Hq, D = q.shape
    G = Hq // cache.k.shape[2]
    scale = 1.0 / math.sqrt(D) if not scale else scale
    out, spread, size = np.zeros((N, Hq, D)), np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for b in range(len(start)):
        lo, n = int(row_offsets[b]), int(row_offsets[b + 1]) - int(row_offsets[b])
        L = int(start[b]) + n
        if not n:
            continue
        k, v = cache.rows(table[b], L)
        back = (int(start[b]) + np.arange(n))[:, None] - np.arange(L)[None, :]
        sees = (back >= 0) & ((back < window) if window else True)
        for h in range(Hq):
            kk, vv = k[:, h // G], v[:, h // G]
            with np.errstate(invalid="ignore"):
                s = np.where(sees, scale * (q[lo:lo + n, h] @ kk.T), -np.inf)
                p = np.exp(s - s.max(axis=1, keepdims=True))
            p = np.where(sees, p, 0.0)
            p /= p.sum(axis=1, keepdims=True)
            out[lo:lo + n, h] = p @ vv
            spread[lo:lo + n, h] = p @ np.abs(vv)
            size[lo:lo + n, h] = np.where(sees, scale * (np.abs(q[lo:lo + n, h]) @ np.abs(kk).T), 0.0).max(axis=1)
    return out, spread, size
