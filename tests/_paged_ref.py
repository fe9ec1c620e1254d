"""Plain 64-bit forms of the paged 8-bit cache's operators (numpy), written from their definitions in
include/tsv_paged.h, one row, page and node at a time."""
import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_values():
    """Value of each of the 256 codes (sign, 4 exponent bits of bias 7, 3 fraction bits; 0x7F and 0xFF are NaN)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = (-1.0 if c & 128 else 1.0), (c >> 3) & 15, c & 7
        out[c] = s * (m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
    out[0x7F] = out[0xFF] = np.nan
    return out


VALUES = e4m3_values()


def round_e4m3(x):
    """Nearest e4m3 value of each x (ties to the even code), saturating; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    with np.errstate(divide="ignore", invalid="ignore"):
        _, e = np.frexp(np.where(a > 0, a, 1.0))
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        r = np.rint(a / step) * step
    return np.where(np.isnan(x), np.nan, np.copysign(np.minimum(r, E4M3_MAX), x))


def scale_for(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    if amax <= 0:
        return 2.0 ** -126
    e = math.ceil(math.log2(amax / E4M3_MAX)) - 1
    while amax > math.ldexp(E4M3_MAX, e):
        e += 1
    return math.ldexp(1.0, max(e, -126))


def need(rows):
    """scale_for of the finite magnitudes of an array."""
    a = np.abs(rows)
    a = a[np.isfinite(a)]
    return scale_for(float(a.max()) if a.size else 0.0)


def rotate(x, positions, inv_freq, interleaved=False, inverse=False, amplitude=1.0):
    """x [N, H, D] -> rotated, in 64 bits (the angle as whole turns taken off exactly in integers)."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(inv_freq)
    for n, p in enumerate(np.asarray(positions).tolist()):
        for i, w in enumerate(np.asarray(inv_freq, dtype=np.float64).tolist()):
            t = math.fmod(p * w, 2 * math.pi) * (-1.0 if inverse else 1.0)
            c, s = amplitude * math.cos(t), amplitude * math.sin(t)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            y[n, :, a] = x[n, :, a] * c - x[n, :, b] * s
            y[n, :, b] = x[n, :, b] * c + x[n, :, a] * s
    return y


class Cache:
    """A cache as values: k, v [pages, rows, Hkv, D] hold the codes' values (value / scale), scales [pages, Hkv]."""

    def __init__(self, k, v, k_scale, v_scale):
        self.k, self.v = np.array(k, dtype=np.float64), np.array(v, dtype=np.float64)
        self.k_scale, self.v_scale = np.array(k_scale, dtype=np.float64), np.array(v_scale, dtype=np.float64)
        self.page = self.k.shape[1]

    def write(self, table_row, start, k_rows, v_rows):
        """New rows (values) behind `start` kept rows of one request."""
        for codes, scales, x in ((self.k, self.k_scale, k_rows), (self.v, self.v_scale, v_rows)):
            done = 0
            while done < len(x):
                at = start + done
                pid, r = int(table_row[at // self.page]), at % self.page
                m = min(self.page - r, len(x) - done)
                for g in range(codes.shape[2]):
                    part = x[done:done + m, g]
                    s = need(part)
                    if r > 0 and done == 0:
                        old = scales[pid, g]
                        s = max(s, old)
                        if s > old:
                            codes[pid, :r, g] = round_e4m3(codes[pid, :r, g] * (old / s))
                    codes[pid, r:r + m, g] = round_e4m3(part / s)
                    scales[pid, g] = s
                done += m

    def rows(self, table_row, count):
        """K and V values [count, Hkv, D] of the first rows of a request's pages."""
        ids = [int(table_row[i // self.page]) for i in range(count)]
        at = [i % self.page for i in range(count)]
        if not count:
            shape = (0,) + self.k.shape[2:]
            return np.zeros(shape), np.zeros(shape)
        return (self.k[ids, at] * self.k_scale[ids][:, :, None], self.v[ids, at] * self.v_scale[ids][:, :, None])


def attention(q, cache, table, prefix_len, node_offsets, tree_table=None, sees=None, scale=None):
    """Returns out [N, Hq, D], and beside it the same sums over |v| (what a relative error of the weights can move)
    and the largest scale * sum |q| |k| over the seen keys [N, Hq].  sees[i, j]: node i (global) sees tree row j; None:
    j <= i within the request."""
    N, Hq, D = q.shape
    G = Hq // cache.k.shape[2]
    scale = 1.0 / math.sqrt(D) if not scale else scale
    out, spread, size = np.zeros((N, Hq, D)), np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for b in range(len(prefix_len)):
        lo, hi = int(node_offsets[b]), int(node_offsets[b + 1])
        P, n = int(prefix_len[b]), hi - lo
        k, v = cache.rows(table[b], P)
        if tree_table is not None:
            tk, tv = cache.rows(tree_table[b], n)
            k, v = np.concatenate([k, tk]), np.concatenate([v, tv])
        for i in range(n):
            see = np.zeros(len(k), dtype=bool)
            see[:P] = True
            if tree_table is not None:
                see[P:] = sees[lo + i, :n] if sees is not None else np.arange(n) <= i
            if not see.any():
                continue
            for h in range(Hq):
                kk, vv = k[see, h // G], v[see, h // G]
                s = scale * (kk @ np.asarray(q[lo + i, h], dtype=np.float64))
                with np.errstate(invalid="ignore"):
                    p = np.exp(s - s.max())
                p /= p.sum()
                out[lo + i, h] = p @ vv
                spread[lo + i, h] = p @ np.abs(vv)
                size[lo + i, h] = (scale * (np.abs(kk) @ np.abs(np.asarray(q[lo + i, h], dtype=np.float64)))).max()
    return out, spread, size


def ancestors(parent, node_offsets):
    """sees[i, j] and the packed words [N, 8] of tree_prepare."""
    N = int(node_offsets[-1])
    sees = np.zeros((N, 256), dtype=bool)
    for b in range(len(node_offsets) - 1):
        lo, hi = int(node_offsets[b]), int(node_offsets[b + 1])
        for i in range(hi - lo):
            j = i
            while j >= 0:
                sees[lo + i, j] = True
                j = int(parent[lo + j])
    words = np.zeros((N, 8), dtype=np.uint32)
    for j in range(256):
        words[:, j >> 5] |= sees[:, j].astype(np.uint32) << np.uint32(j & 31)
    return sees, words.view(np.int32)
