"""Attention of a chunk of new tokens over a paged cache on the GPU, against the 64-bit form of tests/_pages_ref.py.

Tolerance: the bound of test_gpu_paged.py's attention (see _attention_bound there).  The kernels for chunks hold more of a weight
than it allows for (bf16: fp16's 11 bits of it; q to 2^-17 of its row's largest value or better), and fp32 rows on the tensor cores
are held to the bound of the CUDA cores with one addition: q and the weights are two fp16 terms each, off by 2^-22 of themselves."""
import math

import numpy as np
import pytest
import torch

import _pages_ref as P
from test_gpu_paged import HALF_STEP, _attention_bound, dev, i32, make_cache, page_lists, values

pytestmark = pytest.mark.gpu
KINDS = [("f32", torch.float32, 0), ("f32-cuda-cores", torch.float32, 1), ("bf16-cuda-cores", torch.bfloat16, 1),
         ("bf16", torch.bfloat16, 0)]


def bound(ref, spread, size, dtype, keys, D, tensor):
    tol = _attention_bound(ref, spread, size, dtype, keys, D, tensor and dtype == torch.bfloat16)
    return tol + 4 * 2.0 ** -22 * (1 + size[..., None]) * spread if tensor else tol


class Chunk:
    """Random caches, page lists and queries of some requests; lens: (rows in front, new rows) each."""

    def __init__(self, tsv, rng, lens, Hq, Hkv, D, page, dtype=torch.bfloat16, head_major=True, power=True, size=0.4):
        self.lens, self.Hq, self.Hkv, self.D, self.page = lens, Hq, Hkv, D, page
        counts = [-(-(p + n) // page) for p, n in lens]
        self.cache = make_cache(tsv, rng, sum(counts) + 2, page, Hkv, D, head_major, power=power)
        self.table, _ = page_lists(rng, sum(counts) + 2, counts, max(counts) + 1)
        self.start = np.array([p for p, _ in lens])
        self.offs = np.concatenate([[0], np.cumsum([n for _, n in lens])])
        self.q = dev(rng.normal(size=(int(self.offs[-1]), Hq, D)) * size, dtype)
        self.max_rows = max(1, max(n for _, n in lens))

    def run(self, tsv, **kw):
        d = dict(max_rows=self.max_rows)
        d.update(kw)
        return tsv.paged_chunk_attention(self.q, self.cache, dev(self.table), i32(self.start), i32(self.offs), **d)

    def ref(self, window=0, scale=None):
        return P.chunk_attention(self.q.double().cpu().numpy(), values(self.cache), self.table, self.start, self.offs, window, scale)

    def check(self, out, st, flags, window=0, scale=None):
        assert (st.cpu() == 0).all()
        ref, spread, size = self.ref(window, scale)
        got = out.double().cpu().numpy()
        keys = max(p + n for p, n in self.lens)
        tol = bound(ref, spread, size, self.q.dtype, keys, self.D, flags == 0)
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])
        norm = np.linalg.norm(ref)
        if norm:  # errors of single weights are independent: the whole is far nearer than the bound
            assert np.linalg.norm(got - ref) <= (4e-3 if self.q.dtype == torch.bfloat16 else 2e-6) * norm


CASES = [  # page, Hq, Hkv, D, head_major, lengths (rows in front, new rows)
    (16, 4, 4, 128, True, [(0, 1)]),
    (16, 4, 4, 64, True, [(37, 5)]),
    (16, 8, 2, 64, False, [(0, 1), (130, 17), (15, 16), (16, 0), (257, 133)]),
    (32, 3, 1, 128, True, [(128, 20), (127, 1), (129, 3)]),
    (64, 14, 2, 128, False, [(200, 137), (1, 2)]),
    (128, 16, 2, 64, True, [(500, 9), (128, 64)]),
    (128, 8, 1, 128, True, [(300, 100), (0, 300)]),
    (32, 2, 2, 64, True, [(70, 256), (0, 129)]),
    (16, 11, 1, 128, True, [(90, 3), (0, 23)]),
    (64, 70, 1, 128, True, [(150, 2), (0, 9)]),
    (16, 2, 2, 128, True, [(0, 700)]),
    (128, 5, 5, 128, False, [(1000, 257), (0, 128), (127, 2), (128, 128), (511, 1)]),
    (64, 6, 3, 64, True, [(0, 0), (3, 511), (0, 0), (64, 192)]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:5]))
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_chunks(tsv, case, kind):
    page, Hq, Hkv, D, head_major, lens = case
    b = Chunk(tsv, np.random.default_rng(page + Hq), lens, Hq, Hkv, D, page, dtype=kind[1], head_major=head_major)
    ws = tsv.paged_chunk_attention_workspace(b.q, b.cache, len(lens), b.max_rows, flags=kind[2])
    out, st = b.run(tsv, flags=kind[2], workspace=ws)
    b.check(out, st, kind[2])
    again, st = b.run(tsv, flags=kind[2], workspace=ws)
    assert torch.equal(again, out) and (st == 0).all()


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 300, 5000])
@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_windows(tsv, window, kind):
    b = Chunk(tsv, np.random.default_rng(window), [(0, 300), (1000, 1), (333, 140), (64, 64), (700, 17)], 6, 2, 64 if window % 2 else 128,
              32, dtype=kind[1])
    out, st = b.run(tsv, flags=kind[2], window=window)
    b.check(out, st, kind[2], window=window)
    if window == 5000:
        plain, _ = b.run(tsv, flags=kind[2])
        b.check(plain, st, kind[2])


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens(tsv, kind, D):
    """One new token of each request, and of some; with and without a window."""
    lens = [(0, 1), (1, 1), (640, 1), (129, 1), (0, 0), (2000, 1), (127, 1), (5000, 1)]
    b = Chunk(tsv, np.random.default_rng(D), lens, 8, 2, D, 16, dtype=kind[1])
    out, st = b.run(tsv, flags=kind[2])
    b.check(out, st, kind[2])
    wide, st = b.run(tsv, flags=kind[2], max_rows=40)  # more than there are: another kernel may run
    b.check(wide, st, kind[2])
    out, st = b.run(tsv, flags=kind[2], window=130)
    b.check(out, st, kind[2], window=130)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_scale_any_scales_and_strides(tsv, kind):
    """A softmax scale of the caller's; page scales that are no powers of two; a strided q gives the same bits."""
    b = Chunk(tsv, np.random.default_rng(9), [(50, 140), (0, 7), (140, 1), (1300, 290)], 6, 2, 128, 32, dtype=kind[1], power=False)
    out, st = b.run(tsv, flags=kind[2], scale=0.2)
    b.check(out, st, kind[2], scale=0.2)
    q = torch.zeros(b.q.shape[0], b.Hq + 3, b.D + 16, dtype=b.q.dtype, device="cuda")
    q[:, 2:-1, :b.D] = b.q
    b.q = q[:, 2:-1, :b.D]
    again, _ = b.run(tsv, flags=kind[2], scale=0.2)
    assert torch.equal(again, out)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_are_not_seen(tsv, kind, D, window):
    """NaN and huge values behind the last rows, in front of windows and in rows of the chunk itself: only rows that see a
    key get anything from it."""
    rng = np.random.default_rng(11)
    lens = [(37, 160), (300, 5), (0, 3), (130, 300)]
    b = Chunk(tsv, rng, lens, 4, 2, D, 16, dtype=kind[1])
    clean, st = b.run(tsv, flags=kind[2], window=window)
    b.check(clean, st, kind[2], window=window)
    k, v = b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8)
    used = torch.zeros(b.cache.num_pages, 16, dtype=torch.bool, device="cuda")
    for i, (p, n) in enumerate(lens):
        for r in range(max(0, p - window + 1) if window else 0, p + n):
            used[b.table[i][r // 16], r % 16] = True
    k[~used] = 0x7F
    v[~used] = 0xFF
    out, st = b.run(tsv, flags=kind[2], window=window)
    assert torch.equal(out, clean) and (st == 0).all()
    # NaN in V of rows 40, 100 and 196 of request 0, in K of row 302 of request 1, in both ends of the last request's new rows
    want = torch.zeros_like(out, dtype=torch.bool)

    def hit(i, row, heads, dims):
        p, n = lens[i]
        for x in range(n):
            if row <= p + x and (not window or row > p + x - window):
                want[int(b.offs[i]) + x, heads, dims] = True

    for i, row, d in ((0, 40, 5), (0, 100, 6), (0, 196, 7), (3, 130, 1), (3, 429, 2), (3, 200, D - 1)):
        v[b.table[i][row // 16], row % 16, 1, d] = 0x7F
        hit(i, row, slice(2, 4), d)
    k[b.table[1][302 // 16], 302 % 16, 0, 7] = 0xFF
    hit(1, 302, slice(0, 2), slice(None))
    out, st = b.run(tsv, flags=kind[2], window=window)
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], clean[~want])


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_extreme_scores(tsv, kind):
    """Scores of both signs up to thousands, a row of zeros, tiny rows, one of infinities: rows do not touch each other."""
    rng = np.random.default_rng(12)
    b = Chunk(tsv, rng, [(600, 150), (260, 3)], 2, 1, 128, 32, dtype=kind[1])
    b.q[0] *= 60.0
    b.q[1] = 0.0
    b.q[2] *= 1e-6
    b.q[70] *= 1000.0
    out, st = b.run(tsv, flags=kind[2])
    ref, spread, size = b.ref()
    tol = bound(ref, spread, size, b.q.dtype, 750, 128, kind[2] == 0)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    b.q[3], b.q[40] = math.inf, math.nan
    out2, _ = b.run(tsv, flags=kind[2])
    keep = [i for i in range(153) if i not in (3, 40)]
    assert torch.equal(out2[keep], out[keep]) and torch.isnan(out2[3]).all() and torch.isnan(out2[40]).all()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_sink_and_flat_tail(tsv, kind):
    """One key 2^13 times as heavy as each of 6000 equal others, whose sum must not get lost: weights 8192 : 6000."""
    rng = np.random.default_rng(13)
    b = Chunk(tsv, rng, [(5901, 100)], 1, 1, 64, 128, dtype=kind[1])
    k, v = b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8)
    k.zero_()
    v.fill_(0x38)  # 1.0
    b.cache.k_scale.fill_(1.0)
    b.cache.v_scale.fill_(1.0)
    k[b.table[0][3], 77, 0, 0] = 0x38
    v[b.table[0][3], 77] = 0xB8  # -1.0
    b.q.zero_()
    b.q[:, 0, 0] = 13 * math.log(2.0)
    out, _ = b.run(tsv, flags=kind[2], scale=1.0)
    w = math.exp(float(b.q[0, 0, 0].double()))
    n = torch.arange(100, dtype=torch.float64) + 5901
    want = ((n - w) / (n + w))[:, None, None]
    # weights are off by 2^-8 (tensor cores, bf16), the value 1 / 6 by half a step
    tol = (2.0 ** -8 * 1.01 if kind[0] == "bf16" else 6100 * 2.0 ** -23) + HALF_STEP[kind[1]] * want.abs()
    assert ((out.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("where", ["all", "front", "back"])
@pytest.mark.parametrize("page", [16, 128])
def test_pages_of_zero_values(tsv, kind, where, page):
    """V zero in some pages, under the scale that append writes for zeros (2^-126) or a scale of 0: finite, and their weights
    still count."""
    b = Chunk(tsv, np.random.default_rng(14), [(300, 140), (0, 130), (700, 1)], 4, 2, 128, page, dtype=kind[1])
    for scale in (2.0 ** -126, 0.0):
        for i, (p, n) in enumerate(b.lens):
            ids = b.table[i][:-(-(p + n) // page)].tolist()
            half = len(ids) // 2
            ids = torch.tensor({"all": ids, "front": ids[:half], "back": ids[half:]}[where], device="cuda", dtype=torch.int64)
            if scale:
                b.cache.v.view(torch.uint8)[ids, :, 0] = 0
            b.cache.v_scale[ids, 0] = scale
        out, st = b.run(tsv, flags=kind[2])
        b.check(out, st, kind[2])
        if where == "all":
            assert (out[:, :2] == 0).all()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("power", [-126, -110, 100, 115])
def test_a_scale_is_a_factor(tsv, kind, power):
    """V under scales of 2^power (K's stay): the values times 2^power, as far as they are normal numbers.  (Sums over 700 keys of
    values below 2 times 2^127 pass fp32's range before they are divided: the header allows values to 2^127 over the keys.)"""
    b = Chunk(tsv, np.random.default_rng(15), [(300, 140), (0, 130), (700, 1)], 4, 2, 64, 32, dtype=kind[1])
    b.cache.v_scale.fill_(1.0)
    out, st = b.run(tsv, flags=kind[2])
    codes = b.cache.v.view(torch.uint8)
    codes &= 0xBF  # |values| below 2
    out, st = b.run(tsv, flags=kind[2])
    b.cache.v_scale.fill_(2.0 ** power)
    far, st = b.run(tsv, flags=kind[2])
    assert (st == 0).all()
    want = out.double() * 2.0 ** power
    normal = want.abs() >= 2.0 ** -125
    # fp32 results that are turned by a power of two are the same bits; the join of parts may round once more
    tol = 4 * HALF_STEP[kind[1]] if kind[1] == torch.bfloat16 else 2.0 ** -21
    assert ((far.double() - want).abs()[normal] <= tol * want.abs()[normal]).all()
    assert normal.any() or power == -126  # (values below 2, times 2^-126: none is a normal number)
    assert (far.double() - want).abs()[~normal].max().item() <= 2.0 ** -125 if (~normal).any() else True


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("page,D", [(16, 128), (128, 64)])
def test_pages_whose_values_lie_far_apart(tsv, kind, page, D):
    """V scales 2^30 apart from page to page and rows that attend to hardly more than one key: the weights of a page of
    small values are held as well as those of a page of large ones beside it."""
    b = Chunk(tsv, np.random.default_rng(16), [(37, 205), (556, 103), (300, 8), (1800, 1)], 4, 2, D, page, dtype=kind[1])
    pages = torch.arange(b.cache.num_pages, device="cuda")
    b.cache.v_scale.mul_((2.0 ** ((pages * 7) % 31 - 30.0)).unsqueeze(1))
    b.q[::2] *= 60.0  # rows of one key, and flat ones
    out, st = b.run(tsv, flags=kind[2])
    assert (st == 0).all()
    ref, spread, size = b.ref()
    tol = bound(ref, spread, size, b.q.dtype, 1801, D, kind[2] == 0)
    # a weight in fp16 is off by 2^-33 of the row's largest product of weight and scale at the least (codes up to 448); fp32 rows
    # and CUDA cores hold more
    if kind[2] == 0:
        top = spread.max(axis=-1, keepdims=True)
        tol = tol + 2.0 ** -36 * 448 * 4 * top * 16
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), ((err / tol).max(), np.argwhere(err > tol)[:4])


def test_requests_are_rejected_one_by_one(tsv):
    for kind in KINDS:
        rng = np.random.default_rng(17)
        lens = [(40, 30), (10, 40), (70, 5), (0, 20), (90, 9), (33, 50)]
        b = Chunk(tsv, rng, lens, 4, 2, 64, 16, dtype=kind[1])
        good, st = b.run(tsv, flags=kind[2])
        b.check(good, st, kind[2])
        b.table[1, 2] = b.cache.num_pages  # a page id out of range, on each side
        b.table[2, 0] = -1
        b.start[3] = b.table.shape[1] * 16 - 19  # one row more than the list has room for
        b.start[4] = -1
        out, st = b.run(tsv, flags=kind[2], max_rows=49)  # the last request has more rows
        assert st.tolist() == [0, 1, 1, 1, 1, 1]
        assert torch.equal(out[:30], good[:30])
        # rows of no request keep what they hold; offsets that fall, leave q or are negative
        b = Chunk(tsv, rng, [(40, 30), (10, 40)], 4, 2, 64, 16, dtype=kind[1])
        b.offs = np.array([5, 20, 60])
        b.max_rows = 40
        b.start = np.array([4, 10])
        out = torch.full((70, 4, 64), 9.0, dtype=kind[1], device="cuda")
        _, st = b.run(tsv, flags=kind[2], out=out)
        assert st.tolist() == [0, 0] and (out[:5] == 9).all() and (out[60:] == 9).all() and not (out[5:60] == 9).all(-1).any()
        for offs, want in (([0, 71, 70], [1, 1]), ([-1, 10, 20], [1, 0]), ([10, 5, 20], [1, 0]), ([0, 0, 0], [0, 0])):
            b.offs = np.array(offs)
            _, st = b.run(tsv, flags=kind[2], max_rows=100)
            assert st.tolist() == want
        b.start = np.array([2 ** 31 - 1, 2 ** 31 - 20])
        b.offs = np.array([0, 30, 60])
        _, st = b.run(tsv, flags=kind[2])
        assert st.tolist() == [1, 1]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_chunks_of_nothing_and_refusals(tsv, kind):
    b = Chunk(tsv, np.random.default_rng(18), [(5, 0), (0, 0)], 4, 2, 64, 16, dtype=kind[1])
    out, st = b.run(tsv, flags=kind[2])
    assert out.shape == (0, 4, 64) and (st == 0).all()
    b = Chunk(tsv, np.random.default_rng(18), [(5, 3)], 4, 2, 64, 16, dtype=kind[1])
    t, s, o = dev(b.table), i32(b.start), i32(b.offs)
    call = tsv.paged_chunk_attention
    for bad in (lambda: call(b.q[:, :, :32], b.cache, t, s, o), lambda: call(b.q, b.cache, t, s.long(), o),
                lambda: call(b.q, b.cache, t, s, o[:1]), lambda: call(b.q, b.cache, t.t(), s, o),
                lambda: call(b.q, b.cache, t, s, o, out=b.q[:2]), lambda: call(b.q.cpu(), b.cache, t, s, o)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        call(b.q.half(), b.cache, t, s, o)
    for kw in (dict(window=-1), dict(scale=-1.0), dict(flags=2), dict(max_rows=0)):
        with pytest.raises(tsv.TSVError):
            call(b.q, b.cache, t, s, o, **kw)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_captured_chunks_follow_the_lengths(tsv, kind):
    """A captured call reads lengths, lists and cache at the time of its replay; two graphs with workspaces of their own on two
    streams give what eager calls give."""
    rng = np.random.default_rng(41)
    bs = [Chunk(tsv, rng, [(300, 90), (20, 130)], 8, 2, 128, 16, dtype=kind[1]) for _ in range(2)]
    graphs, outs, state = [], [], []
    for b in bs:
        a = dict(table=dev(b.table), start=i32(b.start), offs=i32(b.offs))
        ws = tsv.paged_chunk_attention_workspace(b.q, b.cache, 2, 220, flags=kind[2])
        out, st = torch.empty_like(b.q), torch.zeros(2, dtype=torch.int32, device="cuda")
        call = lambda b=b, a=a, ws=ws, out=out, st=st: tsv.paged_chunk_attention(  # noqa: E731
            b.q, b.cache, a["table"], a["start"], a["offs"], max_rows=220, workspace=ws, out=out, status=st, flags=kind[2])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            call()
            with torch.cuda.graph(g, stream=s):
                call()
        graphs.append((g, s))
        outs.append((out, st))
        state.append(dict(a, ws=ws))  # (a graph's workspace lives as long as the graph)
    for starts, offs in (([300, 20], [0, 90, 220]), ([5, 0], [0, 1, 130]), ([170, 100], [0, 220, 220]), ([0, 149], [0, 0, 1])):
        for a in state:
            a["start"].copy_(i32(starts)), a["offs"].copy_(i32(offs))
        torch.cuda.synchronize()
        for (out, st), (g, s) in zip(outs, graphs):
            out.fill_(3.0)
        torch.cuda.synchronize()
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for b, (out, st) in zip(bs, outs):
            b.start, b.offs, b.lens = np.array(starts), np.array(offs), list(zip(starts, np.diff(offs)))
            eager, st2 = b.run(tsv, flags=kind[2], max_rows=220, out=torch.full_like(b.q, 3.0))
            assert torch.equal(out, eager) and (st == 0).all() and (st2 == 0).all()


def test_a_chunk_on_a_given_stream(tsv):
    b = Chunk(tsv, np.random.default_rng(42), [(300, 90), (20, 130)], 8, 2, 128, 16)
    want, _ = b.run(tsv)
    s = torch.cuda.Stream()
    q = b.q
    b.q = torch.zeros_like(q)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)
        b.q.copy_(q)
    out, st = b.run(tsv, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and (st == 0).all()


LONG = [  # dtype, page, Hq, Hkv, D, lengths, window
    (torch.bfloat16, 16, 8, 1, 128, [(20000, 3)], 0), (torch.bfloat16, 64, 16, 2, 128, [(3000, 1200)], 0),
    (torch.bfloat16, 128, 2, 1, 64, [(0, 2500), (9000, 1), (4000, 33)], 0), (torch.bfloat16, 32, 4, 4, 128, [(5000, 600)], 700),
    (torch.float32, 32, 4, 1, 64, [(9000, 20), (100, 700)], 0), (torch.float32, 128, 8, 2, 128, [(2000, 300), (7000, 1)], 3000),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(str(x) for x in c[1:5]) + str(c[0])[6:])
def test_chunks_over_many_blocks(tsv, case):
    dtype, page, Hq, Hkv, D, lens, window = case
    b = Chunk(tsv, np.random.default_rng(50), lens, Hq, Hkv, D, page, dtype=dtype, size=1.0)
    out, st = b.run(tsv, window=window)
    b.check(out, st, 0, window=window)
    again, _ = b.run(tsv, window=window)
    assert torch.equal(again, out)


MANY = [  # page, Hq, Hkv, D, lengths, window: more units of 256 rows than SMs
    (16, 32, 16, 128, [(300, 1), (0, 257), (9, 1), (200, 400), (0, 1), (1000, 1), (0, 300), (700, 129), (50, 65), (3, 1), (129, 128)], 0),
    (128, 32, 16, 64, [(0, 1)] * 40 + [(5, 700)] + [(600, 1)] * 40 + [(250, 600)], 0),
    (32, 24, 24, 128, [(40, 300), (0, 1), (100, 500), (0, 1), (0, 1), (513, 257), (0, 700)], 150),
    (64, 48, 24, 64, [(1500, 33)] * 20 + [(1000, 200)], 1200),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_many_units_of_one_and_two_tiles(tsv, case):
    page, Hq, Hkv, D, lens, window = case
    b = Chunk(tsv, np.random.default_rng(52), lens, Hq, Hkv, D, page)
    assert -(-len(b.q) * (Hq // Hkv) // 256) * Hkv >= 152
    out, st = b.run(tsv, window=window)
    b.check(out, st, 0, window=window)
    again, _ = b.run(tsv, window=window)
    assert torch.equal(again, out)
    # NaN in V, in masked blocks and others
    v = b.cache.v.view(torch.uint8)
    want = torch.zeros_like(out, dtype=torch.bool)
    G = Hq // Hkv
    for i, (p, n) in enumerate(lens):
        for row, g, d in ((p + n // 2, 1, 3), (p + n - 1, 0, D - 1), (p // 2, Hkv - 1, 0)):
            v[b.table[i][row // page], row % page, g, d] = 0x7F
            for x in range(n):
                if row <= p + x and (not window or row > p + x - window):
                    want[int(b.offs[i]) + x, g * G:(g + 1) * G, d] = True
    got, _ = b.run(tsv, window=window)
    assert torch.equal(torch.isnan(got), want) and torch.equal(got[~want], out[~want])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_largest_batch_of_chunks(tsv, dtype):
    rng = np.random.default_rng(51)
    lens = [(int(p), int(n)) for p, n in zip(rng.integers(0, 300, 128), rng.integers(0, 40, 128))]
    b = Chunk(tsv, rng, lens, 8, 4, 64, 16, dtype=dtype)
    out, st = b.run(tsv)
    b.check(out, st, 0)
    one = Chunk(tsv, rng, [(p, 1) for p, _ in lens], 8, 4, 64, 16, dtype=dtype)
    out, st = one.run(tsv)
    one.check(out, st, 0)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_prompts_in_pieces_fork_and_verification(tsv, kind):
    """A serving loop over its operators: pages taken, a prompt appended and attended to in pieces, samples forked from it (their
    last page copied), single tokens, a page list cut back, the pool compacted with the pages' contents moved, and the same
    attention as before: each step against plain arithmetic on what the cache holds."""
    rng = np.random.default_rng(60)
    _, dtype, flags = kind
    page, Hq, Hkv, D, slots, width, num = 16, 4, 2, 64, 6, 20, 100
    cache = tsv.PagedCache.empty(num, page, Hkv, D)
    pool = tsv.PagePool(num)
    table, held = torch.full((slots, width), -1, dtype=torch.int32, device="cuda"), i32([0] * slots)
    freq, _ = tsv.rope_frequencies(D, device="cuda")
    new = lambda n, h: dev(rng.normal(size=(n, h, D)), dtype)  # noqa: E731
    length = np.zeros(slots, dtype=int)

    def tokens(counts):
        """New tokens of every slot: pages, rows, attention, checked."""
        nonlocal length
        st = tsv.pages_resize(pool, table, held, i32(length + counts), page)
        assert (st == 0).all()
        offs = np.concatenate([[0], np.cumsum(counts)])
        N = int(offs[-1])
        pos = np.concatenate([length[b] + np.arange(counts[b]) for b in range(slots)])
        q = tsv.rope(new(N, Hq), i32(pos), freq)
        st = tsv.paged_append(cache, table, new(N, Hkv), new(N, Hkv), i32(offs), start=i32(length), positions=i32(pos), inv_freq=freq)
        assert (st == 0).all()
        out, st = tsv.paged_chunk_attention(q, cache, table, i32(length), i32(offs), max_rows=int(max(counts)), flags=flags)
        assert (st == 0).all()
        ref, spread, size = P.chunk_attention(q.double().cpu().numpy(), values(cache), table.tolist(), length, offs)
        tol = bound(ref, spread, size, dtype, 400, D, flags == 0)
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
        start, length = length.copy(), length + counts
        return q, start, offs, out

    tokens(np.array([100, 33, 0, 0, 0, 0]))  # two prompts, the first piece
    tokens(np.array([50, 0, 0, 0, 0, 0]))    # the second piece of one
    f = tsv.pages_fork(pool, table[:2], held[:2], i32([0, 0, 1, 0]), i32([150, 150, 33, 96]), table[2:], held[2:], page)
    assert f["status"].tolist() == [0] * 4
    assert tsv.pages_copy(cache, f["copy_src"], f["copy_dst"]).tolist() == [0]
    length[2:] = [150, 150, 33, 96]
    before = values(cache)
    t = table.tolist()
    for b, s in ((2, 0), (3, 0), (4, 1), (5, 0)):  # the children hold what their sources hold
        for x, y in zip(before.rows(t[b], length[b]), before.rows(t[s], length[b])):
            assert np.array_equal(x, y)
    for _ in range(3):
        tokens(np.array([1, 1, 1, 1, 0, 1]))
    q, start, offs, out = tokens(np.array([7, 0, 40, 1, 3, 20]))
    # sample 3 ends, sample 5 goes back to 80 rows, which end with a whole page
    length[3], length[5] = 0, 80
    assert (tsv.pages_resize(pool, table, held, i32(length), page) == 0).all()
    live = int((pool.refs > 0).sum())
    c = tsv.pages_compact(pool, [table], [held], in_place=True)
    assert (c["status"] == 0).all() and int((pool.refs[:live] > 0).sum()) == live and (pool.refs[live:] == 0).all()
    assert tsv.pages_copy(cache, c["move_src"], c["move_dst"], count=c["moved"]).tolist() == [0]
    keep = [0, 1, 2, 4]
    rows = np.concatenate([np.arange(offs[b], offs[b + 1]) for b in keep])
    again, st = tsv.paged_chunk_attention(q[rows].contiguous(), cache, table[keep].contiguous(), i32(start[keep]),
                                          i32(np.concatenate([[0], np.cumsum(np.diff(offs)[keep])])), max_rows=40, flags=flags)
    assert (st == 0).all()
    # the same rows in other pages; where a unit's work is cut may differ
    tol = 2 * HALF_STEP[dtype] * out[rows].double().abs() + (2.0 ** -10 if dtype == torch.bfloat16 else 2.0 ** -18)
    assert ((again.double() - out[rows].double()).abs() <= tol).all()
    # nothing holds a page that no list holds
    count = torch.zeros(num, dtype=torch.int32, device="cuda")
    for b in range(slots):
        ids = table[b, :int(held[b])].long()
        count.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    assert torch.equal(count, pool.refs)
