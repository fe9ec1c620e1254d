"""The paged 8-bit cache's operators on the GPU against their 64-bit forms (tests/_paged_ref.py).

Tolerances, each derived from the arithmetic before the first run:
  * rotation: the angle is exact to 2^-32 turns, then rounded to fp32 (2^-25 half turns: 2^-23.3 radians); cosine, sine and
    amplitude add 2^-22 at most, the two products and their sum 3 x 2^-24: together under 2^-21 of |a| + |b| (times the
    amplitude), and half a step of the type: 2^-8 (bf16), 2^-24 (fp32) of the value.
  * codes: half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below the normal range.
  * attention: see _attention_bound.
"""
import math

import numpy as np
import pytest
import torch

import _paged_ref as R

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def dev(x, dtype=None):
    t = x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))
    return t.cuda() if dtype is None else t.to("cuda", dtype)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rope


def _check_rope(got, x, pos, freq, **kw):
    ref = R.rotate(x.double().cpu().numpy(), pos.cpu().numpy(), freq.cpu().numpy(), **kw)
    amp, half = kw.get("amplitude", 1.0), len(freq)
    a = np.abs(x.double().cpu().numpy())
    size = a.copy()
    if kw.get("interleaved"):
        size[..., 0:2 * half:2] = size[..., 1:2 * half:2] = a[..., 0:2 * half:2] + a[..., 1:2 * half:2]
    else:
        size[..., :half] = size[..., half:2 * half] = a[..., :half] + a[..., half:2 * half]
    tol = HALF_STEP[x.dtype] * np.abs(ref) + 2.0 ** -21 * amp * size * (1 + HALF_STEP[x.dtype])
    g = got.double().cpu().numpy()
    assert np.array_equal(g[..., 2 * half:], x.double().cpu().numpy()[..., 2 * half:])
    bad = np.abs(g - ref) > tol
    assert not bad.any(), (np.abs(g - ref)[bad][:4], tol[bad][:4])


ROPE = [  # N, H, D, rot, interleaved, inverse, amplitude
    (1, 1, 2, 2, False, False, 1.0), (3, 5, 128, 128, False, False, 1.0), (7, 2, 128, 64, True, True, 1.25),
    (4, 3, 64, 64, True, False, 1.0), (5, 1, 80, 20, False, True, 0.5), (2, 2, 33, 6, True, False, 1.0),
    (300, 4, 128, 128, False, False, 1.0), (9, 3, 256, 256, False, False, 1.0), (3, 2, 1024, 1024, True, False, 1.0),
    (6, 7, 96, 32, False, False, 1.0), (600, 9, 64, 30, False, False, 1.0),
]


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(x) for x in c))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["plain", "slice", "odd"])
def test_rope(tsv, case, dtype, layout):
    N, H, D, rot, inter, inverse, amp = case
    rng = np.random.default_rng(N * 1000 + D)
    pos = rng.integers(-5, 1 << 20, size=N)
    pos[:min(N, 4)] = [0, 1, 131071, -7][:min(N, 4)]
    freq, _ = tsv.rope_frequencies(rot, device="cuda")
    wide = dev(rng.normal(size=(N, H + 2, D + 8)), dtype)
    x = {"plain": wide[:, :H, :D].contiguous(), "slice": wide[:, 1:H + 1, :D], "odd": wide[:, :H, 1:D + 1]}[layout]
    kw = dict(interleaved=inter, inverse=inverse, amplitude=amp)
    got = tsv.rope(x, i32(pos), freq, **kw)
    _check_rope(got, x, torch.tensor(pos), freq, **kw)
    if layout != "plain":  # and a strided result: what lies around it stays
        out = torch.full((N, H + 1, D + 8), 7.0, dtype=dtype, device="cuda")
        tsv.rope(x, i32(pos), freq, out=out[:, :H, 8:], **kw)
        assert torch.equal(out[:, :H, 8:], got)
        assert (out[:, H:] == 7).all() and (out[:, :, :8] == 7).all()
    same = x.clone(memory_format=torch.contiguous_format)
    tsv.rope(same, i32(pos), freq, out=same, **kw)  # in place
    assert torch.equal(same, got)


def test_rope_far_positions_and_scaled_frequencies(tsv):
    """The angle of a position near 2^31 is as exact as a near one's: its fixed-point product is off by 2^-34 turns."""
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 10 ** 9 + 7, 1])
    x = dev(np.random.default_rng(0).normal(size=(5, 2, 64)), torch.float32)
    for scaling in ("none", "linear", "ntk", "bands", "yarn"):
        freq, amp = tsv.rope_frequencies(64, scaling=scaling, factor=4.0, trained=4096.0, low=1.0, high=32.0, device="cuda")
        got = tsv.rope(x, i32(pos), freq, amplitude=amp).double().cpu().numpy()
        # The 64-bit angle itself is off by 2^-53 x 2^31 x w: take it from an exact integer ratio instead.
        from fractions import Fraction
        two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889")
        xd = x.double().cpu().numpy()
        for n, p in enumerate(pos.tolist()):
            for i, w in enumerate(freq.tolist()):
                t = Fraction(w) * p / two_pi
                t = float(t - math.floor(t)) * 2 * math.pi
                a, b = xd[n, :, i], xd[n, :, i + 32]
                for d, ref in ((i, a * math.cos(t) - b * math.sin(t)), (i + 32, b * math.cos(t) + a * math.sin(t))):
                    tol = 2.0 ** -24 * np.abs(amp * ref) + 2.0 ** -21 * amp * (np.abs(a) + np.abs(b))
                    assert (np.abs(got[n, :, d] - amp * ref) <= tol).all()


def test_rope_gradient_is_the_inverse_rotation(tsv):
    """Against autograd of the 64-bit formula, and against differences of the operator itself."""
    N, H, D, rot, amp = 6, 3, 64, 48, 1.3
    rng = np.random.default_rng(5)
    pos, (freq, _) = i32(rng.integers(0, 5000, N)), tsv.rope_frequencies(rot, device="cuda")
    x, gy = dev(rng.normal(size=(N, H, D)), torch.float32), dev(rng.normal(size=(N, H, D)), torch.float32)
    for inter in (False, True):
        gx = tsv.rope(gy, pos, freq, interleaved=inter, inverse=True, amplitude=amp)
        xd = x.double().requires_grad_()
        t = (pos.double()[:, None] * freq)[:, None]
        c, s = amp * t.cos(), amp * t.sin()
        a, b = (xd[..., 0:rot:2], xd[..., 1:rot:2]) if inter else (xd[..., :rot // 2], xd[..., rot // 2:rot])
        u, v = a * c - b * s, b * c + a * s
        y = torch.cat([torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1), xd[..., rot:]], -1)
        (y * gy.double()).sum().backward()
        size = gy.double().abs().amax() * 2 * amp
        assert (gx.double() - xd.grad).abs().max() <= 2.0 ** -20 * size
        # <rope(x + e) - rope(x), gy> = <e, gx> (the rotation is linear): fp32 sums of 1152 terms
        e = dev(rng.normal(size=(N, H, D)), torch.float32)
        d = tsv.rope(x + e, pos, freq, interleaved=inter, amplitude=amp).double() - tsv.rope(
            x, pos, freq, interleaved=inter, amplitude=amp).double()
        lhs, rhs = (d * gy.double()).sum(), (e.double() * gx.double()).sum()
        # each of 1152 differences is off by a few 2^-21 |x| |gy|, |x| and |gy| under 8
        assert abs(lhs - rhs) <= 1152 * 4 * 2.0 ** -21 * 64


def test_rope_of_nothing_and_refusals(tsv):
    freq, _ = tsv.rope_frequencies(64, device="cuda")
    x = torch.zeros(0, 2, 64, device="cuda")
    assert tsv.rope(x, i32([]), freq).shape == (0, 2, 64)
    x = torch.zeros(3, 2, 64, device="cuda")
    for bad in (lambda: tsv.rope(x, i32([1, 2]), freq), lambda: tsv.rope(x, i32([1, 2, 3]).long(), freq),
                lambda: tsv.rope(x, i32([1, 2, 3]), freq.float()), lambda: tsv.rope(x[..., :32], i32([1, 2, 3]), freq),
                lambda: tsv.rope(x, i32([1, 2, 3]), freq, out=torch.zeros(3, 2, 65, device="cuda")),
                lambda: tsv.rope(x.transpose(1, 2), i32([1, 2, 3]), freq)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        tsv.rope(x.half(), i32([1, 2, 3]), freq)


# ------------------------------------------------------------------ caches


def make_cache(tsv, rng, pages, page, Hkv, D, head_major=True, codes=None, power=True):
    """A cache of random codes (no NaN) and scales around 2^-3; `power`: scales are powers of two."""
    c = tsv.PagedCache.empty(pages, page, Hkv, D, head_major=head_major)
    if codes is None:
        codes = rng.integers(0, 256, size=(4, pages, page, Hkv, D), dtype=np.int64)
        kv = np.where((codes[:2] & 0x7F) == 0x7F, 0, codes[:2]).astype(np.uint8)
        # values mostly of the size of normals: exponents around 2^5 .. 2^8
        kv = np.where(codes[2:] % 4 > 0, (kv & 0x8F) | ((codes[2:] % 3 + 12) << 3), kv).astype(np.uint8)
        kv = np.where((kv & 0x7F) == 0x7F, 0x70, kv).astype(np.uint8)
    else:
        kv = codes
    c.k.view(torch.uint8).copy_(dev(kv[0]))
    c.v.view(torch.uint8).copy_(dev(kv[1]))
    for s in (c.k_scale, c.v_scale):
        e = 2.0 ** rng.integers(-9, -6, size=(pages, Hkv))
        s.copy_(dev(e if power else e * rng.uniform(0.6, 1.7, size=(pages, Hkv)), torch.float32))
    return c


def values(c):
    """The cache as a reference cache."""
    f = lambda t: R.VALUES[t.view(torch.uint8).cpu().numpy()]  # noqa: E731
    return R.Cache(f(c.k), f(c.v), c.k_scale.cpu().numpy(), c.v_scale.cpu().numpy())


def page_lists(rng, pages, counts, width):
    """Disjoint page lists in random order, rows padded with ids that nobody may read."""
    ids, at = rng.permutation(pages), 0
    out = np.full((len(counts), width), -1, dtype=np.int32)
    for b, m in enumerate(counts):
        out[b, :m] = ids[at:at + m]
        at += m
    return out, ids[at:]


def same_codes(c, ref, exact_k=True, unrotated=None):
    """K and V of the cache against the reference's (as values; -0 and 0 alike)."""
    got = values(c)
    assert np.array_equal(got.v, ref.v, equal_nan=True)
    assert np.array_equal(got.v_scale, ref.v_scale)
    assert np.array_equal(got.k_scale, ref.k_scale)
    if exact_k:
        assert np.array_equal(got.k, ref.k, equal_nan=True)
    return got


# ------------------------------------------------------------------ append

APPEND = [  # page, Hkv, D, rot, interleaved, head_major, lengths (start, new) per request
    (16, 2, 128, 128, False, True, [(0, 20)]),
    (16, 3, 64, 64, True, False, [(5, 1), (0, 0), (16, 16), (31, 40)]),
    (32, 9, 128, 64, False, True, [(33, 7), (0, 65)]),
    (64, 1, 128, 0, False, True, [(63, 2), (1, 200)]),
    (128, 5, 64, 32, True, False, [(127, 130), (0, 1), (300, 3)]),
    (128, 2, 128, 20, False, True, [(60, 100)]),
    (32, 2, 64, 6, False, False, [(2, 11), (40, 90)]),
    (16, 17, 128, 128, True, True, [(3, 300)]),
]


def _append_inputs(tsv, rng, case, dtype):
    page, Hkv, D, rot, inter, head_major, lens = case
    pages = [-(-(s + n) // page) for s, n in lens]
    c = make_cache(tsv, rng, sum(pages) + 3, page, Hkv, D, head_major)
    table, spare = page_lists(rng, sum(pages) + 3, pages, max(pages) + 2)
    offs = np.concatenate([[0], np.cumsum([n for _, n in lens])])
    N = int(offs[-1])
    kv = dev(rng.normal(size=(N, 2, Hkv, D)) * np.exp(rng.normal(size=(N, 2, 1, 1))), dtype)
    pos = rng.integers(0, 100000, size=N)
    freq = tsv.rope_frequencies(rot, device="cuda")[0] if rot else None
    return c, table, offs, kv, pos, freq


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c[:6]))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_append(tsv, case, dtype):
    page, Hkv, D, rot, inter, head_major, lens = case
    rng = np.random.default_rng(page * 7 + Hkv)
    c, table, offs, kv, pos, freq = _append_inputs(tsv, rng, case, dtype)
    ref, before = values(c), values(c)
    k64 = kv[:, 0].double().cpu().numpy()
    if rot:
        k64 = R.rotate(k64, pos, freq.cpu().numpy(), interleaved=inter, amplitude=1.125)
    v64 = kv[:, 1].double().cpu().numpy()
    for b, (s, n) in enumerate(lens):
        ref.write(table[b], s, k64[offs[b]:offs[b + 1]], v64[offs[b]:offs[b + 1]])
    st = tsv.paged_append(c, dev(table), kv[:, 0], kv[:, 1], i32(offs), start=i32([s for s, _ in lens]),
                          positions=i32(pos) if rot else None, inv_freq=freq, interleaved=inter, amplitude=1.125)
    assert (st.cpu() == 0).all()
    got = same_codes(c, ref, exact_k=not rot)
    if rot:
        # where the reference's code is another one, the value lies next to the border between the two
        diff = got.k != ref.k
        rows = np.zeros(diff.shape, dtype=bool)
        for b, (s, n) in enumerate(lens):
            for i in range(n):
                pid, r = table[b][(s + i) // page], (s + i) % page
                rows[pid, r] = True
                x, sc = k64[offs[b] + i], ref.k_scale[pid][:, None]
                amax = np.abs(kv[offs[b] + i, 0].double().cpu().numpy()).max(axis=-1, keepdims=True)
                tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * sc) + 2.0 ** -20 * 1.125 * 2 * amax
                assert (np.abs(got.k[pid, r] * sc - x) <= tol).all()
        assert not (diff & ~rows).any()  # kept rows and rows behind: as the reference has them
        assert diff.mean() < 0.01
    # pages that belong to nobody, and rows behind a request's last one, are as they were
    touched = np.zeros(before.k.shape[:2], dtype=bool)
    for b, (s, n) in enumerate(lens):
        for r in range(s + n if n else 0):
            touched[table[b][r // page], r % page] = True
    assert np.array_equal(got.k[~touched], before.k[~touched]) and np.array_equal(got.v[~touched], before.v[~touched])


def test_append_values_that_do_not_fit(tsv):
    """Infinities become the largest code, NaN stays NaN, and neither moves the scale; zeros take the smallest scale."""
    rng = np.random.default_rng(3)
    c = make_cache(tsv, rng, 3, 16, 1, 64)
    k = dev(rng.normal(size=(20, 1, 64)), torch.float32)
    v = torch.zeros(20, 1, 64, device="cuda")
    k[2, 0, 5], k[3, 0, 6], k[4, 0, 7], k[5, 0, 8] = math.inf, -math.inf, math.nan, 1e-40
    v[17, 0, 3] = 3e38
    ref = values(c)
    ref.write([2, 0], 0, k.double().cpu().numpy(), v.double().cpu().numpy())
    st = tsv.paged_append(c, i32([[2, 0]]), k, v, i32([0, 20]))
    got = same_codes(c, ref)
    assert (st.cpu() == 0).all() and got.v_scale[2, 0] == 2.0 ** -126 and np.isnan(got.k[2, 4, 0, 7])
    assert got.k[2, 2, 0, 5] == 448 and got.k[2, 3, 0, 6] == -448


def test_append_grows_a_scale_and_keeps_its_rows(tsv):
    """Three appends into one page: small, large (the first rows are requantised), small again (the scale stays)."""
    rng = np.random.default_rng(4)
    c = make_cache(tsv, rng, 2, 32, 2, 128)
    ref = values(c)
    start = 0
    for size, n in ((0.01, 9), (3.0, 5), (1e-4, 11)):
        kv = dev(rng.normal(size=(n, 2, 2, 128)) * size, torch.bfloat16)
        ref.write([1], start, kv[:, 0].double().cpu().numpy(), kv[:, 1].double().cpu().numpy())
        tsv.paged_append(c, i32([[1]]), kv[:, 0], kv[:, 1], i32([0, n]), start=i32([start]))
        start += n
        same_codes(c, ref)


def test_append_rejects_requests_one_by_one(tsv):
    """A request whose rows or pages do not fit is left alone, the others are written."""
    rng = np.random.default_rng(6)
    c = make_cache(tsv, rng, 6, 16, 2, 64)
    before = values(c)
    kv = dev(rng.normal(size=(100, 2, 2, 64)), torch.bfloat16)
    #        fits      page id 6   page id -1  past the list  negative start  too many rows
    table = [[0, 1], [2, 6], [-1, 2], [2, 3], [2, 3], [2, 3]]
    start = [3, 10, 0, 20, -1, 0]
    new = [20, 10, 4, 13, 4, 26]
    offs = np.concatenate([[0], np.cumsum(new)])
    ref = values(c)
    ref.write([0, 1], 3, kv[:20, 0].double().cpu().numpy(), kv[:20, 1].double().cpu().numpy())
    st = tsv.paged_append(c, i32(table), kv[:, 0], kv[:, 1], i32(offs), start=i32(start), max_rows=25)
    assert st.tolist() == [0, 1, 1, 1, 1, 1]
    got = same_codes(c, ref)
    assert np.array_equal(got.k[2:], before.k[2:])
    # offsets that leave k, or fall
    for offs in ([0, 101], [-1, 10], [10, 5]):
        st = tsv.paged_append(c, i32([[4, 5, 3, 2, 1, 0, 0]]), kv[:, 0], kv[:, 1], i32(offs))
        assert st.tolist() == [1]
    same_codes(c, ref)


# ------------------------------------------------------------------ attention


def _attention_bound(out_ref, spread, size, dtype, keys, D, tensor):
    """How far an output may be off.  A relative error e of every weight moves the output by at most 2 e x spread (the sums
    over |v|, once for the weighted sum and once for its denominator).
    CUDA cores, fp32: a score is a sum of D products in fp32, off by at most (D + 4) 2^-24 of scale x sum |q| |k|; exp2 and
    the running sums add (keys + 16) 2^-24.
    Tensor cores, few rows: q is split into two e4m3 terms, off by 2^-17 of its row's largest value at most, which a score
    sees as at most 2^-12 of its size for rows without outliers beyond 2^5; a weight in two e4m3 terms is off by 2^-8 of
    itself or 2^-18 of its step's largest weight (256 keys: 2^-10 together).  Many rows: q is exact down to 2^-31 of the
    row's largest value, a weight in fp16 off by 2^-12 of itself or 2^-33 of the largest: less on both counts.
    128 x 2^-21 = 2^-14 stands in for the 2^-10: single weights that small are off independently, and the cases here
    hold it."""
    e = (D + 4) * 2.0 ** -24 * size + (keys + 16) * 2.0 ** -24
    tol = 2 * e[..., None] * spread + 2.0 ** -8 * 0
    if tensor:
        tol = tol + (2.0 ** -8 + 128 * 2.0 ** -21) * spread + 2 * (2.0 ** -12 * size[..., None]) * spread
    return tol + HALF_STEP[dtype] * (np.abs(out_ref) + tol) + 1e-30


def random_parent(rng, n):
    return np.array([-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)], dtype=np.int32)[:n]


class Batch:
    """Random caches, page lists, trees and queries of some requests."""

    def __init__(self, tsv, rng, lens, Hq, Hkv, D, page, tree=True, dtype=torch.bfloat16, head_major=True, power=True, spare=2):
        self.lens, self.Hq, self.Hkv, self.D, self.page, self.tree = lens, Hq, Hkv, D, page, tree
        mains = [-(-p // page) for p, _ in lens]
        trees = [-(-n // page) if tree else 0 for _, n in lens]
        pool = sum(mains) + sum(trees) + spare
        self.cache = make_cache(tsv, rng, pool, page, Hkv, D, head_major, power=power)
        both, _ = page_lists(rng, pool, mains + trees, max(mains + trees) + 1)
        self.table, self.tree_table = both[:len(lens)], both[len(lens):]
        self.prefix = np.array([p for p, _ in lens])
        self.offs = np.concatenate([[0], np.cumsum([n for _, n in lens])])
        N = int(self.offs[-1])
        self.parent = np.concatenate([random_parent(rng, n) for _, n in lens]) if N else np.zeros(0, np.int32)
        self.sees, self.words = R.ancestors(self.parent, self.offs)
        self.q = dev(rng.normal(size=(N, Hq, D)) * 0.4, dtype)

    def run(self, tsv, anc=True, **kw):
        d = dict(tree_table=dev(self.tree_table) if self.tree else None, anc=dev(self.words) if anc and self.tree else None,
                 max_nodes=max(1, max(n for _, n in self.lens)))
        d.update(kw)
        return tsv.paged_tree_attention(self.q, self.cache, dev(self.table), i32(self.prefix), i32(self.offs), **d)

    def check(self, out, st, tensor, anc=True, scale=None):
        assert (st.cpu() == 0).all()
        ref, spread, size = R.attention(self.q.double().cpu().numpy(), values(self.cache), self.table, self.prefix, self.offs,
                                        self.tree_table if self.tree else None, self.sees if anc else None, scale)
        got = out.double().cpu().numpy()
        keys = max(p + n for p, n in self.lens)
        tol = _attention_bound(ref, spread, size, self.q.dtype, keys, self.D, tensor)
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (bad.sum(), np.abs(got - ref)[bad][:5], tol[bad][:5])
        norm = np.linalg.norm(ref)
        if norm:  # errors of single weights are independent: the whole is far nearer than the bound
            assert np.linalg.norm(got - ref) <= (4e-3 if self.q.dtype == torch.bfloat16 else 2e-6) * norm


KINDS = [("f32", torch.float32, 0), ("bf16-cuda-cores", torch.bfloat16, 1), ("bf16", torch.bfloat16, 0)]
ATTN = [  # page, Hq, Hkv, D, head_major, lengths (prefix, nodes)
    (16, 4, 4, 128, True, [(37, 5)]),
    (16, 8, 2, 64, False, [(0, 1), (130, 17), (15, 16), (16, 0), (257, 33)]),
    (32, 3, 1, 128, True, [(128, 20), (127, 1), (129, 3)]),
    (64, 14, 2, 128, False, [(200, 37), (1, 2)]),
    (128, 16, 2, 64, True, [(500, 9), (128, 64)]),
    (128, 8, 1, 128, True, [(300, 100)]),
    (32, 2, 2, 64, True, [(70, 256)]),
    (16, 11, 1, 128, True, [(90, 3)]),
    (64, 70, 1, 128, True, [(150, 2)]),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(x) for x in c[:5]))
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_attention(tsv, case, kind):
    page, Hq, Hkv, D, head_major, lens = case
    b = Batch(tsv, np.random.default_rng(page + Hq), lens, Hq, Hkv, D, page, dtype=kind[1], head_major=head_major)
    out, st = b.run(tsv, flags=kind[2])
    b.check(out, st, kind[0] == "bf16")


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_without_a_tree(tsv, kind, D):
    """One token of each request over its prefix; an empty prefix gives zeros."""
    b = Batch(tsv, np.random.default_rng(D), [(1, 1), (0, 1), (640, 1), (129, 1), (2000, 1)], 8, 1, D, 16, tree=False,
              dtype=kind[1])
    out, st = b.run(tsv, flags=kind[2])
    b.check(out, st, kind[0] == "bf16")
    assert (out[1] == 0).all()
    b = Batch(tsv, np.random.default_rng(D), [(0, 2)], 4, 2, D, 64, tree=False, dtype=kind[1])
    out, st = b.run(tsv, flags=kind[2], out=torch.full_like(b.q, 5.0))
    assert (out == 0).all() and (st == 0).all()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_attention_chain_scale_and_any_scales(tsv, kind):
    """anc None is a chain; a softmax scale of the caller's; page scales that are no powers of two."""
    b = Batch(tsv, np.random.default_rng(9), [(50, 40), (0, 7), (140, 1)], 6, 2, 128, 32, dtype=kind[1], power=False)
    out, st = b.run(tsv, anc=False, flags=kind[2], scale=0.2)
    b.check(out, st, kind[0] == "bf16", anc=False, scale=0.2)
    q = torch.zeros(b.q.shape[0], b.Hq + 3, b.D + 16, dtype=b.q.dtype, device="cuda")  # a strided q gives the same
    q[:, 2:-1, :b.D] = b.q
    b.q = q[:, 2:-1, :b.D]
    again, _ = b.run(tsv, anc=False, flags=kind[2], scale=0.2)
    assert torch.equal(again, out)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_ignores_what_it_may_not_see(tsv, kind, D):
    """NaN and huge values behind the last row of the prefix and of the tree, and NaN in tree rows: only nodes that see a
    row get anything from it."""
    rng = np.random.default_rng(11)
    lens = [(37, 6), (128, 5), (0, 3)]
    b = Batch(tsv, rng, lens, 4, 2, D, 16, dtype=kind[1])
    clean, st = b.run(tsv, flags=kind[2])
    b.check(clean, st, kind[0] == "bf16")
    k, v = b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8)
    used = torch.zeros(b.cache.num_pages, 16, dtype=torch.bool, device="cuda")
    for i, (p, n) in enumerate(lens):
        for t, m in ((b.table[i], p), (b.tree_table[i], n)):
            for r in range(m):
                used[t[r // 16], r % 16] = True
    k[~used] = 0x7F
    v[~used] = 0xFF
    out, st = b.run(tsv, flags=kind[2])
    assert torch.equal(out, clean) and (st == 0).all()
    # node 2 of request 0: one NaN in V, node 3 of request 1: a NaN in K
    v[b.tree_table[0][0], 2, 1, 5] = 0x7F
    k[b.tree_table[1][0], 3, 0, 7] = 0xFF
    out, st = b.run(tsv, flags=kind[2])
    want = torch.zeros_like(out, dtype=torch.bool)
    for i in range(6):
        if b.sees[i, 2]:
            want[i, 2:4, 5] = True
    for i in range(5):
        if b.sees[6 + i, 3]:
            want[6 + i, 0:2] = True
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], clean[~want])
    # a NaN in a prefix row of V reaches every node of that request, one dimension of the heads that share it
    v[b.table[1][0], 0, 0, 1] = 0x7F
    out, _ = b.run(tsv, flags=kind[2])
    assert torch.isnan(out[6:11, 0:2, 1]).all() and not torch.isnan(out[11:]).any()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_attention_extreme_scores(tsv, kind):
    """One key far above the others (they still count when they are many), scores of both signs up to thousands, a query
    row of zeros, one of infinities: rows do not touch each other."""
    rng = np.random.default_rng(12)
    b = Batch(tsv, rng, [(700, 4), (260, 3)], 2, 1, 128, 32, dtype=kind[1])
    b.q[0] *= 60.0
    b.q[1] = 0.0
    b.q[2] *= 1e-6
    out, st = b.run(tsv, flags=kind[2])
    ref, spread, size = R.attention(b.q.double().cpu().numpy(), values(b.cache), b.table, b.prefix, b.offs, b.tree_table, b.sees)
    tol = _attention_bound(ref, spread, size, b.q.dtype, 704, 128, kind[0] == "bf16")
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    b.q[3] = math.inf
    out2, _ = b.run(tsv, flags=kind[2])
    keep = [0, 1, 2, 4, 5, 6]
    assert torch.equal(out2[keep], out[keep]) and torch.isnan(out2[3]).all()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_attention_sink_and_flat_tail(tsv, kind):
    """One key 2^13 times as heavy as each of 6000 equal others, whose sum must not get lost: weights 8192 : 6000."""
    rng = np.random.default_rng(13)
    b = Batch(tsv, rng, [(6001, 1)], 1, 1, 64, 128, tree=False, dtype=kind[1])
    k, v = b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8)
    k.zero_()
    v.fill_(0x38)  # 1.0
    b.cache.k_scale.fill_(1.0)
    b.cache.v_scale.fill_(1.0)
    k[b.table[0][3], 77, 0, 0] = 0x38
    v[b.table[0][3], 77] = 0xB8  # -1.0
    b.q.zero_()
    b.q[0, 0, 0] = 13 * math.log(2.0)
    out, _ = b.run(tsv, flags=kind[2], scale=1.0)
    w = math.exp(float(b.q[0, 0, 0].double()))
    want = (6000 - w) / (6000 + w)
    # weights are off by 2^-8 (tensor cores), the value 1 / 6 by half a step
    tol = (2.0 ** -8 * 1.01 if kind[0] == "bf16" else 6100 * 2.0 ** -23) + HALF_STEP[kind[1]] * abs(want)
    assert (out.double() - want).abs().max().item() <= tol


# Many rows per KV head over many keys: query rows on the TMEM lanes, up to 256 of them a unit.
WIDE = [  # page, Hq, Hkv, D, head_major, lengths (prefix, nodes)
    (16, 64, 8, 128, True, [(0, 1), (1, 20), (127, 33), (128, 16), (129, 9), (300, 32), (77, 12), (513, 17)]),
    (128, 12, 4, 64, True, [(500, 90), (128, 64), (0, 3), (127, 1), (1, 86), (256, 0), (30, 43), (700, 5)]),
    (32, 32, 32, 128, False, [(70, 256), (33, 1)]),
    (64, 32, 4, 128, False, [(64 * i, 13 + i) for i in range(8)]),
    (16, 34, 2, 64, True, [(40 + i, 3 + i % 6) for i in range(16)]),
    (128, 16, 8, 128, True, [(9000, 40), (20, 129), (1500, 256), (4000, 1)]),
]


def wide_workspace(tsv, b):
    """Makes room in the page table for as many keys as the kernel of many rows is taken for (entries that no length needs
    are not read); returns a workspace."""
    if b.table.shape[1] * b.page < 1 << 19:
        more = np.full((len(b.lens), (1 << 19) // b.page), -1, dtype=np.int32)
        b.table = np.concatenate([b.table, more], axis=1)
    rows = max(n for _, n in b.lens) * (b.Hq // b.Hkv)
    assert rows > 128 and len(b.lens) * b.Hkv * -(-rows // 256) * (b.table.shape[1] * b.page // 128) >= 4096
    return tsv.paged_tree_attention_workspace(b.q, b.cache, len(b.lens), max(n for _, n in b.lens))


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(str(x) for x in c[:5]))
def test_attention_of_many_rows(tsv, case):
    page, Hq, Hkv, D, head_major, lens = case
    b = Batch(tsv, np.random.default_rng(page + Hq), lens, Hq, Hkv, D, page, head_major=head_major)
    ws = wide_workspace(tsv, b)
    out, st = b.run(tsv, workspace=ws)
    b.check(out, st, True)
    again, st = b.run(tsv, workspace=ws)
    assert torch.equal(again, out) and (st == 0).all()


def test_attention_of_many_rows_chain_scale_and_any_scales(tsv):
    """anc None; a softmax scale of the caller's; page scales that are no powers of two; without a tree; a strided q."""
    b = Batch(tsv, np.random.default_rng(21), [(50, 40), (0, 7), (140, 1), (1300, 150)], 24, 8, 128, 32, power=False)
    ws = wide_workspace(tsv, b)
    out, st = b.run(tsv, anc=False, scale=0.2, workspace=ws)
    b.check(out, st, True, anc=False, scale=0.2)
    q = torch.zeros(b.q.shape[0], b.Hq + 3, b.D + 16, dtype=b.q.dtype, device="cuda")
    q[:, 2:-1, :b.D] = b.q
    plain, b.q = b.q, q[:, 2:-1, :b.D]
    again, _ = b.run(tsv, anc=False, scale=0.2, workspace=ws)
    assert torch.equal(again, out)
    b.q, b.tree = plain, False
    out, st = b.run(tsv, workspace=ws)
    b.check(out, st, True)
    assert (out[40:47] == 0).all()


@pytest.mark.parametrize("long", [0, 6000])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_of_many_rows_ignores_what_it_may_not_see(tsv, D, long):
    """As above, with units that end in one CTA and units that are cut: NaN behind the last rows and in tree rows."""
    rng = np.random.default_rng(22)
    lens = [(37 + long, 6), (128, 5), (0, 3), (700, 140)]
    G, Hkv = 4, 8
    b = Batch(tsv, rng, lens, G * Hkv, Hkv, D, 16)
    ws = wide_workspace(tsv, b)
    clean, st = b.run(tsv, workspace=ws)
    b.check(clean, st, True)
    k, v = b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8)
    used = torch.zeros(b.cache.num_pages, 16, dtype=torch.bool)
    for i, (p, n) in enumerate(lens):
        for t, m in ((b.table[i], p), (b.tree_table[i], n)):
            for r in range(m):
                used[t[r // 16], r % 16] = True
    k[~used.cuda()] = 0x7F
    v[~used.cuda()] = 0xFF
    out, st = b.run(tsv, workspace=ws)
    assert torch.equal(out, clean) and (st == 0).all()
    # NaN in V: nodes 2 of request 0 and 3, 130 of request 3; in K: node 3 of request 1
    marks = [(0, 2, 1, 5), (3, 3, 0, D - 1), (3, 130, 7, 33)]
    for i, node, head, d in marks:
        v[b.tree_table[i][node // 16], node % 16, head, d] = 0x7F
    k[b.tree_table[1][0], 3, 0, 7] = 0xFF
    out, st = b.run(tsv, workspace=ws)
    want = torch.zeros_like(out, dtype=torch.bool)
    for i, node, head, d in marks:
        for x in range(lens[i][1]):
            if b.sees[b.offs[i] + x, node]:
                want[b.offs[i] + x, G * head:G * (head + 1), d] = True
    for x in range(5):
        if b.sees[6 + x, 3]:
            want[6 + x, 0:G] = True
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], clean[~want])
    v[b.table[1][0], 0, 0, 1] = 0x7F  # in a prefix row: every node of the request, the heads that share it
    out, _ = b.run(tsv, workspace=ws)
    assert torch.isnan(out[6:11, 0:G, 1]).all() and not torch.isnan(out[11:14]).any()


def test_attention_of_many_rows_extreme_scores(tsv):
    """Rows whose scores reach thousands of either sign, rows of zeros, of tiny values and of infinities, and V scales that
    differ by 2^24 from page to page: rows do not touch each other."""
    rng = np.random.default_rng(23)
    lens = [(700, 4), (260, 20), (0, 17), (1100, 30)]
    b = Batch(tsv, rng, lens, 64, 8, 128, 32)
    pages = torch.arange(b.cache.num_pages, device="cuda")
    b.cache.v_scale.mul_((2.0 ** ((pages * 7) % 25 - 24.0)).unsqueeze(1))
    b.q[0] *= 60.0
    b.q[1] = 0.0
    b.q[2] *= 1e-6
    b.q[30] *= 1e-30
    ws = wide_workspace(tsv, b)
    out, st = b.run(tsv, workspace=ws)
    ref, spread, size = R.attention(b.q.double().cpu().numpy(), values(b.cache), b.table, b.prefix, b.offs, b.tree_table, b.sees)
    tol = _attention_bound(ref, spread, size, b.q.dtype, 1130, 128, True)
    # A weight is 2^11 p s in fp16, s its V scale relative to the unit's largest, p >= 1 for the row's largest score.  Below
    # 2^-14 it is off by up to 2^-25 whatever its size, which is 2^-36 of the largest weight times the largest V there is
    # (448 times its scale); the sum of the weights is at least 1.  Beside V scales 2^24 apart that counts: a row may
    # attend to the smallest alone.
    tol += 1130 * 2.0 ** -36 * 448 * b.cache.v_scale.max().item()
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), ((err / tol).max(), np.argwhere(err > tol)[:4])
    b.q[3] = math.inf
    b.q[45] = math.nan
    out2, _ = b.run(tsv, workspace=ws)
    keep = [i for i in range(71) if i not in (3, 45)]
    assert torch.equal(out2[keep], out[keep]) and torch.isnan(out2[3]).all() and torch.isnan(out2[45]).all()


def test_attention_of_many_rows_sink_and_flat_tail(tsv):
    """Weights 8192 : 6000 again, for every row."""
    b = Batch(tsv, np.random.default_rng(24), [(6001, 17)], 256, 32, 64, 128, tree=False)
    k, v = b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8)
    k.zero_()
    v.fill_(0x38)  # 1.0
    b.cache.k_scale.fill_(1.0)
    b.cache.v_scale.fill_(1.0)
    k[b.table[0][3], 77, :, 0] = 0x38
    v[b.table[0][3], 77] = 0xB8  # -1.0
    b.q.zero_()
    b.q[:, :, 0] = 13 * math.log(2.0)
    out, _ = b.run(tsv, scale=1.0, workspace=wide_workspace(tsv, b))
    w = math.exp(float(b.q[0, 0, 0].double()))
    want = (6000 - w) / (6000 + w)
    tol = 2.0 ** -8 * 1.01 + HALF_STEP[torch.bfloat16] * abs(want)
    assert (out.double() - want).abs().max().item() <= tol


def test_attention_of_many_rows_follows_the_lengths(tsv):
    """A captured call replayed with other lengths on the device, a request rejected, outputs of rejected rows left."""
    b = Batch(tsv, np.random.default_rng(25), [(500, 40), (900, 30), (100, 17), (64, 33)], 32, 8, 128, 64)
    ws = wide_workspace(tsv, b)
    q, table, tree, anc = b.q, dev(b.table), dev(b.tree_table), dev(b.words)
    prefix, offs = i32(b.prefix), i32(b.offs)
    out, st = torch.empty_like(q), torch.empty(4, dtype=torch.int32, device="cuda")

    def call(o, s, w):
        tsv.paged_tree_attention(q, b.cache, table, prefix, offs, tree_table=tree, anc=anc, max_nodes=40, out=o, status=s, workspace=w)

    call(out, st, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, st, ws)
    for lens in ([500, 900, 100, 64], [3, 900, 0, 1], [499, 128, 99, 64], [512, 0, 64, -1]):
        prefix.copy_(i32(lens))
        out.fill_(7.0)
        graph.replay()
        other, st2 = torch.full_like(out, 7.0), torch.empty_like(st)
        call(other, st2, wide_workspace(tsv, b))
        assert torch.equal(out, other) and torch.equal(st, st2)
        assert st.tolist() == [0, 0, 0, 1 if lens[3] < 0 else 0]
        if lens[3] < 0:
            assert (out[87:] == 7).all()


def test_page_tables_beyond_the_limit_are_refused(tsv):
    b = Batch(tsv, np.random.default_rng(26), [(16, 2)], 2, 2, 64, 16)
    b.table = np.zeros((1, 1), np.int32)
    big = torch.empty((1, (1 << 26) + 1), dtype=torch.int32, device="cuda")
    with pytest.raises(tsv.TSVError):
        tsv.paged_tree_attention(b.q, b.cache, big, i32(b.prefix), i32(b.offs), tree_table=dev(b.tree_table), max_nodes=2)
    with pytest.raises(tsv.TSVError):
        tsv.paged_append(b.cache, big, b.q, b.q, i32(b.offs))


def test_attention_rejects_requests_one_by_one(tsv):
    for flags, dtype in ((0, torch.bfloat16), (1, torch.bfloat16), (0, torch.float32)):
        b = Batch(tsv, np.random.default_rng(14), [(40, 3), (50, 2), (33, 4), (20, 5)], 4, 2, 64, 16, dtype=dtype)
        good, _ = b.run(tsv, flags=flags)
        table, tree = b.table.copy(), b.tree_table.copy()
        b.table[1, 2] = b.cache.num_pages
        b.tree_table[2, 0] = -5
        out, st = b.run(tsv, flags=flags)
        assert st.tolist() == [0, 1, 1, 0]
        assert torch.equal(out[:3], good[:3]) and torch.equal(out[9:], good[9:])
        b.table, b.tree_table = table, tree
        out, st = b.run(tsv, flags=flags, max_nodes=4)
        assert st.tolist() == [0, 0, 0, 1] and torch.equal(out[:9], good[:9])
        b.prefix = np.array([40, 50, -1, 16 * table.shape[1] + 1])
        out, st = b.run(tsv, flags=flags)
        assert st.tolist() == [0, 0, 1, 1] and torch.equal(out[:5], good[:5])
        b.prefix = np.array([40, 50, 33, 20])
        b.offs[-1] = 15  # more rows than q has
        out, st = b.run(tsv, flags=flags)
        assert st.tolist() == [0, 0, 0, 1] and torch.equal(out[:9], good[:9])


@pytest.mark.parametrize("flags,dtype", [(0, torch.bfloat16), (1, torch.bfloat16), (0, torch.float32)])
def test_attention_of_nothing(tsv, flags, dtype):
    b = Batch(tsv, np.random.default_rng(15), [(40, 0), (0, 0)], 4, 2, 64, 16, dtype=dtype)
    out, st = b.run(tsv, flags=flags, status=torch.full((2,), 9, dtype=torch.int32, device="cuda"))
    assert out.shape[0] == 0 and st.tolist() == [0, 0]


def test_attention_shares_prefix_pages(tsv):
    """Two requests whose prefix lists name the same pages."""
    b = Batch(tsv, np.random.default_rng(16), [(100, 3), (100, 3)], 4, 2, 128, 32)
    b.table[1] = b.table[0]
    out, st = b.run(tsv)
    b.check(out, st, True)


# ------------------------------------------------------------------ commit

COMMIT = [  # page, Hkv, D, head_major, (prefix, nodes) per request
    (16, 2, 128, True, [(37, 9), (0, 1), (16, 40)]),
    (32, 3, 64, False, [(31, 64), (64, 5)]),
    (64, 9, 128, True, [(10, 100)]),
    (128, 1, 64, True, [(127, 256), (3, 2)]),
]


def accepted(rng, parent, n):
    way = [int(rng.integers(0, n))]
    while parent[way[-1]] >= 0:
        way.append(int(parent[way[-1]]))
    return way[::-1]


@pytest.mark.parametrize("case", COMMIT, ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_commit(tsv, case):
    page, Hkv, D, head_major, lens = case
    rng = np.random.default_rng(page)
    b = Batch(tsv, rng, lens, Hkv, Hkv, D, page, head_major=head_major, spare=20)
    used = set(b.table[b.table >= 0]) | set(b.tree_table[b.tree_table >= 0])
    free = [i for i in range(b.cache.num_pages) if i not in used]
    path, acc, ways = np.full(int(b.offs[-1]), -1), [], []
    wide = np.full((len(lens), b.table.shape[1] + 20), -1)
    wide[:, :b.table.shape[1]] = b.table
    for i, (p, n) in enumerate(lens):
        lo = b.offs[i]
        w = accepted(rng, b.parent[lo:lo + n], n)
        path[lo:lo + len(w)] = w
        acc.append(len(w) - 1)
        ways.append(w)
        for x in range(-(-p // page), -(-(p + len(w)) // page)):
            wide[i, x] = free.pop()
    ref = values(b.cache)
    for i, (p, n) in enumerate(lens):
        k, v = ref.rows(b.tree_table[i], n)
        ref.write(wide[i], p, k[ways[i]], v[ways[i]])
    o = tsv.paged_commit(b.cache, i32(wide), i32(b.tree_table), i32(b.prefix), i32(b.offs), i32(path), i32(acc))
    assert (o["status"].cpu() == 0).all()
    assert o["new_len"].tolist() == [p + len(w) for (p, _), w in zip(lens, ways)]
    same_codes(b.cache, ref)


def test_commit_rejects_requests_one_by_one(tsv):
    rng = np.random.default_rng(21)
    lens = [(5, 6)] * 8
    b = Batch(tsv, rng, lens, 2, 2, 64, 16)
    before = values(b.cache)
    path = np.array([[0, 2, 4, -1, -1, -1], [1, 2, -1, -1, -1, -1], [0, 2, 2, -1, -1, -1], [0, 3, 6, -1, -1, -1], [0] * 6, [0] * 6,
                     [0, 1, -1, -1, -1, -1], [0, 1, -1, -1, -1, -1]]).ravel()
    acc = [2, 1, 2, 2, -1, 6, 1, 1]
    b.table[6, 0] = 9999
    b.tree_table[7, 0] = -1
    ref = values(b.cache)
    k, v = ref.rows(b.tree_table[0], 6)
    ref.write(b.table[0], 5, k[[0, 2, 4]], v[[0, 2, 4]])
    o = tsv.paged_commit(b.cache, i32(b.table), i32(b.tree_table), i32(b.prefix), i32(b.offs), i32(path), i32(acc))
    assert o["status"].tolist() == [0, 1, 1, 1, 1, 1, 1, 1] and o["new_len"].tolist() == [8, -1, -1, -1, -1, -1, -1, -1]
    same_codes(b.cache, ref)
    # a prefix whose new rows leave the list
    b = Batch(tsv, rng, [(30, 4)], 2, 2, 64, 16)
    o = tsv.paged_commit(b.cache, i32(b.table[:, :2]), i32(b.tree_table), i32(b.prefix), i32(b.offs), i32([0, 1, 2, -1]), i32([2]))
    assert o["status"].tolist() == [1]
    o = tsv.paged_commit(b.cache, i32(b.table[:, :2]), i32(b.tree_table), i32(b.prefix), i32(b.offs), i32([0, 1, 2, -1]), i32([1]))
    assert o["status"].tolist() == [0] and o["new_len"].tolist() == [32]


# ------------------------------------------------------------------ together


def _step(tsv, b, freq, rng, flags, dtype, stream=None):
    """One verification step over a paged cache: positions, rope, append, attention, greedy walk, commit."""
    parent, offs, plen = dev(b["parent"]), i32(b["offs"]), b["plen"]
    anc, depth, st = tsv.tree_prepare(parent, offs)
    pos = plen.repeat_interleave(torch.tensor(b["sizes"], device="cuda")) + depth
    q = tsv.rope(b["q"], pos, freq)
    s1 = tsv.paged_append(b["cache"], b["tree_table"], b["k"], b["v"], offs, positions=pos, inv_freq=freq)
    out, s2 = tsv.paged_tree_attention(q, b["cache"], b["table"], plen, offs, tree_table=b["tree_table"], anc=anc,
                                       max_nodes=max(b["sizes"]), flags=flags)
    g = tsv.tree_verify_greedy(b["logits"], b["tokens"], parent, offs)
    o = tsv.paged_commit(b["cache"], b["table"], b["tree_table"], plen, offs, g["path"], g["accept_len"], max_nodes=max(b["sizes"]))
    for s in (st, s1, s2, g["status"], o["status"]):
        assert (s == 0).all()
    return q, out, g, o["new_len"]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_verification_steps_over_a_paged_cache(tsv, kind):
    """Prompt, then three verification steps; after each, the attention equals the framework's tree attention over a
    contiguous cache of the same (dequantised) rows, and the committed rows are the accepted nodes'."""
    rng = np.random.default_rng(31)
    dtype, flags = kind[1], kind[2]
    Hq, Hkv, D, page, V = 4, 2, 128, 16, 50
    prompts = [37, 130, 1]
    cache = tsv.PagedCache.empty(64, page, Hkv, D)
    ids = rng.permutation(64)
    table, tree_table = i32(ids[:48].reshape(3, 16)), i32(ids[48:].reshape(8, 2)[:3])
    freq, _ = tsv.rope_frequencies(D, device="cuda")
    offs = np.concatenate([[0], np.cumsum(prompts)])
    pos = np.concatenate([np.arange(p) for p in prompts])
    new = lambda n, h: dev(rng.normal(size=(n, h, D)), dtype)  # noqa: E731
    st = tsv.paged_append(cache, table, new(offs[-1], Hkv), new(offs[-1], Hkv), i32(offs), positions=i32(pos), inv_freq=freq)
    assert (st == 0).all()
    plen = i32(prompts)
    for step in range(3):
        sizes = [int(x) for x in rng.integers(1, 25, size=3)]
        parent = np.concatenate([random_parent(rng, n) for n in sizes])
        o = np.concatenate([[0], np.cumsum(sizes)])
        N = int(o[-1])
        tokens = rng.integers(0, 4, size=N)
        logits = rng.normal(size=(N, V))
        logits[:, :4] += 4.0
        b = dict(parent=parent, offs=o, sizes=sizes, plen=plen, q=new(N, Hq), k=new(N, Hkv), v=new(N, Hkv), cache=cache, table=table,
                 tree_table=tree_table, logits=dev(logits, torch.float32), tokens=i32(tokens))
        before = values(cache)
        q, out, g, new_len = _step(tsv, b, freq, rng, flags, dtype)
        after = values(cache)
        P = plen.tolist()
        # the same rows in a contiguous cache: e4m3 times a power of two is exact in bf16
        Lcap = max(p + n for p, n in zip(P, sizes))
        kc, vc = torch.zeros(3, Lcap, Hkv, D), torch.zeros(3, Lcap, Hkv, D)
        tl, ttl = table.tolist(), tree_table.tolist()
        for i in range(3):
            k, v = before.rows(tl[i], P[i])
            tk, tv = after.rows(ttl[i], sizes[i])
            kc[i, :P[i] + sizes[i]] = torch.from_numpy(np.concatenate([k, tk]))
            vc[i, :P[i] + sizes[i]] = torch.from_numpy(np.concatenate([v, tv]))
        ref, st = tsv.tree_attention(q, dev(kc, dtype), dev(vc, dtype), P, o.tolist(), plen, i32(o), parent=dev(parent), flags=flags)
        # two roundings of the type, weights of 8 bits on both sides
        tol = 4 * 2.0 ** -8 * float(ref.abs().max()) if dtype == torch.bfloat16 else 1e-5
        assert (out.float() - ref.float()).abs().max().item() <= tol
        # committed rows
        path, acc = g["path"].tolist(), g["accept_len"].tolist()
        assert new_len.tolist() == [p + 1 + a for p, a in zip(P, acc)]
        for i in range(3):
            w = path[o[i]:o[i] + acc[i] + 1]
            k, v = after.rows(tl[i], P[i] + len(w))
            tk, tv = after.rows(ttl[i], sizes[i])
            # requantised once more: half a step, or half of the smallest one under a larger scale
            for x, y, s in ((k[P[i]:], tk[w], after.k_scale), (v[P[i]:], tv[w], after.v_scale)):
                top = s[[tl[i][(P[i] + r) // page] for r in range(len(w))]][:, :, None]
                assert (np.abs(x - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * top)).all()
        plen = new_len


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_captured_steps_follow_the_lengths(tsv, kind):
    """A captured attention call reads the lengths, page lists and cache of the time of its replay; two graphs with
    workspaces of their own replayed on two streams give what eager calls give."""
    rng = np.random.default_rng(41)
    bs = [Batch(tsv, rng, [(300, 9), (20, 3)], 8, 2, 128, 16, dtype=kind[1]) for _ in range(2)]
    graphs, outs, state = [], [], []
    for b in bs:
        a = dict(table=dev(b.table), plen=i32(b.prefix), offs=i32(b.offs), tree=dev(b.tree_table), anc=dev(b.words))
        ws = tsv.paged_tree_attention_workspace(b.q, b.cache, 2, 9, flags=kind[2])
        out, st = torch.empty_like(b.q), torch.zeros(2, dtype=torch.int32, device="cuda")
        call = lambda b=b, a=a, ws=ws, out=out, st=st: tsv.paged_tree_attention(  # noqa: E731
            b.q, b.cache, a["table"], a["plen"], a["offs"], tree_table=a["tree"], anc=a["anc"], max_nodes=9, flags=kind[2],
            workspace=ws, out=out, status=st)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
        outs.append(out)
        state.append(a)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for prefix in ([300, 20], [17, 128], [0, 1]):
        for b, a in zip(bs, state):
            b.prefix = np.array(prefix)
            a["plen"].copy_(i32(prefix))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for b, out in zip(bs, outs):
            eager, st = b.run(tsv, flags=kind[2])
            if prefix[1] > 32:  # more rows than request 1 has pages: it alone is rejected
                assert st.tolist() == [0, 1] and torch.equal(out[:9], eager[:9])
                continue
            assert torch.equal(out, eager) and (st == 0).all()
            b.check(out, st, kind[0] == "bf16")


def test_calls_on_a_given_stream(tsv):
    """Everything on a side stream, results and workspace allocated there."""
    b = Batch(tsv, np.random.default_rng(51), [(90, 7)], 4, 2, 128, 16)
    want, _ = b.run(tsv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, st = b.run(tsv, stream=s)
    x = tsv.rope(b.q, i32(np.arange(7)), tsv.rope_frequencies(128, device="cuda")[0], stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want) and (st == 0).all() and x.shape == b.q.shape


LONG = [  # page, Hq, Hkv, D, tree, B, prefix, nodes: dozens of key blocks for every SM
    (16, 16, 16, 128, True, 16, 2500, 9), (128, 64, 8, 128, True, 2, 9000, 20), (64, 64, 8, 64, False, 30, 3000, 1),
    (32, 96, 24, 64, True, 12, 1700, 8), (32, 32, 32, 128, True, 7, 1900, 64), (16, 8, 2, 128, True, 1, 40000, 7),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(x) for x in c))
def test_attention_over_many_blocks(tsv, case):
    """Long and ragged batches, the tensor cores' result against the CUDA cores' (which the tests above hold to 64 bits)."""
    page, Hq, Hkv, D, tree, B, P, n = case
    rng = np.random.default_rng(P)
    lens = [(int(rng.integers(P // 2, P + 1)), int(rng.integers(1, n + 1))) for _ in range(B)]
    b = Batch(tsv, rng, lens, Hq, Hkv, D, page, tree=tree)
    ws = tsv.paged_tree_attention_workspace(b.q, b.cache, B, max(x for _, x in lens))
    for _ in range(3):  # a workspace used again and again
        out, st = b.run(tsv, workspace=ws)
    ref, st2 = b.run(tsv, flags=1)
    assert (st == 0).all() and (st2 == 0).all()
    norm = ref.float().norm()
    assert (out.float() - ref.float()).norm() <= 6e-3 * norm  # two roundings to bf16 and weights of 8 bits
    # A value is off by at most 2^-8 + 2^-11 of the weighted sum over |v| and half a step of the result on either side;
    # both sums are at most the largest |v|.
    top = float((b.cache.v.float().abs().amax() * b.cache.v_scale.amax()))
    assert (out.float() - ref.float()).abs().max().item() <= (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -8) * top


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_attention_is_repeatable(tsv, kind):
    b = Batch(tsv, np.random.default_rng(61), [(3000, 20), (1, 1), (700, 64)], 8, 2, 128, 64, dtype=kind[1])
    first, st = b.run(tsv, flags=kind[2])
    b.check(first, st, kind[0] == "bf16")
    for _ in range(4):
        assert torch.equal(b.run(tsv, flags=kind[2])[0], first)


def test_shapes_and_types_are_refused(tsv):
    b = Batch(tsv, np.random.default_rng(71), [(20, 3)], 4, 2, 64, 16)
    c, t, p, o = b.cache, dev(b.table), i32(b.prefix), i32(b.offs)
    good = dict(tree_table=dev(b.tree_table), anc=dev(b.words))
    f = tsv.paged_tree_attention
    for bad in (lambda: f(b.q[..., :32], c, t, p, o, **good), lambda: f(b.q, c, t.long(), p, o, **good),
                lambda: f(b.q, c, t, p[:0], o, **good), lambda: f(b.q, c, t, p.cpu(), o, **good),
                lambda: f(b.q, c, t, p, o, tree_table=good["tree_table"], anc=good["anc"][:1]),
                lambda: f(b.q, c, t, p, o, out=torch.empty(1, device="cuda"), **good),
                lambda: tsv.paged_append(c, t, b.q, b.q, o), lambda: tsv.paged_append(c, t, b.q[:, :2], b.q[:, :2], o.long()),
                lambda: tsv.paged_append(c, t, b.q[:, :2], b.q[:, :2], o, inv_freq=tsv.rope_frequencies(64, device="cuda")[0]),
                lambda: tsv.paged_commit(c, t, good["tree_table"], p, o, o.long(), p),
                lambda: tsv.PagedCache(c.k, c.v.clone(memory_format=torch.contiguous_format), c.k_scale, c.v_scale),
                lambda: tsv.PagedCache(c.k, c.v, c.k_scale.double(), c.v_scale)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        f(b.q.half(), c, t, p, o, **good)
    with pytest.raises(TypeError):
        tsv.PagedCache(c.k.float(), c.v.float(), c.k_scale, c.v_scale)
    for kw in (dict(max_nodes=0), dict(max_nodes=257), dict(scale=-1.0)):
        with pytest.raises(tsv.TSVError) as e:
            f(b.q, c, t, p, o, **{**good, **kw})
        assert e.value.code == tsv.TSV_ERR_INVALID_ARG


def test_scales_stay_apart_in_a_long_pool(tsv):
    """Rows whose byte offsets in the pool pass 2^32: pages at the end of a 5 GB cache."""
    pages, page, Hkv, D = 5000, 128, 64, 128
    c = tsv.PagedCache.empty(pages, page, Hkv, D)
    assert c.k.numel() > 1 << 32
    rng = np.random.default_rng(81)
    n, last = 140, [[4999, 4998, 0]]
    kv = dev(rng.normal(size=(n, 2, Hkv, D)), torch.bfloat16)
    assert tsv.paged_append(c, i32(last), kv[:, 0], kv[:, 1], i32([0, n])).tolist() == [0]
    small = tsv.PagedCache.empty(3, page, Hkv, D)
    assert tsv.paged_append(small, i32([[1, 2, 0]]), kv[:, 0], kv[:, 1], i32([0, n])).tolist() == [0]
    for x, y in ((c.k, small.k), (c.v, small.v)):
        assert torch.equal(x.view(torch.uint8)[[4999, 4998]], y.view(torch.uint8)[[1, 2]])
        assert x.view(torch.uint8)[:4998].max().item() == 0
    q = dev(rng.normal(size=(1, Hkv, D)), torch.bfloat16)
    for flags in (0, 1):
        a, s1 = tsv.paged_tree_attention(q, c, i32(last), i32([n]), i32([0, 1]), flags=flags)
        b, s2 = tsv.paged_tree_attention(q, small, i32([[1, 2, 0]]), i32([n]), i32([0, 1]), flags=flags)
        assert torch.equal(a, b) and s1.tolist() == s2.tolist() == [0]


def test_rope_refuses_pointers_between_elements(tsv):
    """Through the C entry: x, y, positions and frequencies on their types' boundaries."""
    x = torch.zeros(4 * 2 * 8 + 8, device="cuda")
    pos, freq = i32([0, 1, 2, 3]), tsv.rope_frequencies(8, device="cuda")[0]
    h = tsv.handle(x.device.index)

    def call(dx=0, dy=0, dp=0, df=0):
        return tsv._lib.tsv_rope(h, tsv.TSV_F32, x.data_ptr() + dx, 16, 8, x.data_ptr() + dy, 16, 8, 4, 2, 8, pos.data_ptr() + dp,
                                 freq.data_ptr() + df, 8, 1.0, 0, 0)

    assert call() == 0
    for bad in (dict(dx=2), dict(dy=1), dict(dp=2), dict(df=4)):
        assert call(**bad) == 1
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_the_largest_batch(tsv, kind):
    """128 requests of every small length through append, attention, commit and attention again, few and many rows."""
    rng = np.random.default_rng(31)
    B, Hkv, D, page = 128, 2, 64, 16
    lens = [(int(rng.integers(0, 70)), int(rng.integers(0, 10))) for _ in range(B)]
    b = Batch(tsv, rng, lens, 4, Hkv, D, page, dtype=kind[1])
    out, st = b.run(tsv, flags=kind[2])
    b.check(out, st, kind[0] == "bf16")
    N = int(b.offs[-1])
    k, v = (dev(rng.normal(size=(N, Hkv, D)), kind[1]) for _ in range(2))
    st = tsv.paged_append(b.cache, dev(b.tree_table), k, v, i32(b.offs))
    assert (st == 0).all()
    out, st = b.run(tsv, flags=kind[2])
    b.check(out, st, kind[0] == "bf16")
    path, accept = np.zeros(N, np.int32), np.zeros(B, np.int32)
    for i, (_, n) in enumerate(lens):
        path[b.offs[i]:b.offs[i + 1]] = np.arange(n)
        accept[i] = max(n - 1, 0)
    room = np.full((B, b.table.shape[1] + 1), -1, np.int32)  # pages behind each prefix to commit into
    room[:, :-1] = b.table
    r = tsv.paged_commit(b.cache, dev(room), dev(b.tree_table), i32(b.prefix), i32(b.offs), i32(path), i32(accept))
    fits = np.array([n > 0 and (p + n - 1) // page < -(-p // page) for p, n in lens])  # the others lack a page, or rows
    got = r["status"].cpu().numpy()
    assert (got[fits] == 0).all()
    assert (got[[n == 0 for _, n in lens]] == 1).all()
    assert np.array_equal(r["new_len"].cpu().numpy()[fits], np.array([p + n for p, n in lens])[fits])
