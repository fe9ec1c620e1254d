"""Chunk attention on the GPU where a page's scale, or what a page outside a row's sight holds, decides: values are code x scale, and
nothing but the rows that a token sees counts.  Bounds as in test_gpu_paged_chunk.py unless a test derives its own."""
import numpy as np
import pytest
import torch

from test_gpu_paged_chunk import KINDS, Chunk
from test_gpu_paged_chunk_range import MIXED

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


def _flat(tsv, dtype, lens, page=16, D=64):
    """A batch of one head whose keys all score 0 but row 3, which scores q's first element; all V are 1, row 3's is 0."""
    b = Chunk(tsv, np.random.default_rng(8), lens, 1, 1, D, page, dtype=dtype)
    k, v = b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8)
    k.zero_()
    v.fill_(0x38)
    b.cache.k_scale.fill_(1.0)
    b.cache.v_scale.fill_(1.0)
    b.q.zero_()
    for i in range(len(lens)):
        k[b.table[i][0], 3, 0, 0] = 0x38
        v[b.table[i][0], 3] = 0
    return b


# What a weight is off by, at most: fp16's half step on the tensor cores (chunks in bf16), two terms of it (fp32: 2^-22), fp32's
# exp2 and products otherwise.
WEIGHT = {"f32": 2.0 ** -21, "f32-cuda-cores": 2.0 ** -22, "bf16-cuda-cores": 2.0 ** -22, "bf16": 2.0 ** -11}


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_weights_hold_fp16s_bits(tsv, kind):
    """n equal weights against one that is about as heavy as all of them (V 1 and -1): every weight is off the same way, so that a
    single rounding shows, and the result is near 0, where its own rounding does not hide it.  One unit, not cut."""
    b = _flat(tsv, kind[1], [(560, 40)])
    b.cache.v.view(torch.uint8)[b.table[0][0], 3] = 0xB8
    b.q[:, 0, 0] = 6.375
    n = 560 + torch.arange(40, dtype=torch.float64)
    worst = 0.0
    for scale in np.linspace(0.985, 1.02, 36).astype(np.float32):
        out, st = b.run(tsv, flags=kind[2], scale=float(scale))
        assert (st == 0).all()
        w = float(np.exp(6.375 * np.float64(scale)))
        want = (n - w) / (n + w)
        # the score (6.4, a few roundings of 2^-24 each: 2^-20), the weights, sums of 38 steps (2^-18), the result's half step
        tol = (WEIGHT[kind[0]] * n + 2.0 ** -20 * w) / (n + w) + 2.0 ** -18 + (2.0 ** -8 if kind[1] == torch.bfloat16 else 2.0 ** -24) * want.abs()
        err = (out[:, 0].double().cpu() - want[:, None]).abs()
        worst = max(worst, (err / tol[:, None]).max().item())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("power", range(10, 38, 3))
def test_light_weights_beside_a_heavy_one(tsv, kind, power):
    """n weights 2^-power of another, whose V is 0: they are all of the result.  In fp16 a weight is off by 2^-33 of the row's
    largest at the most beside its half step; fp32 rows hold theirs to 2^-38 of 16 keys' largest."""
    b = _flat(tsv, kind[1], [(560, 40)])
    b.q[:, 0, 0] = power * np.log(2.0)
    out, st = b.run(tsv, flags=kind[2], scale=1.0)
    assert (st == 0).all()
    n = (560 + torch.arange(40, dtype=torch.float64))[:, None]
    w = np.exp(float(b.q[0, 0, 0].double()))
    want = n / (n + w)
    floor = {"bf16": 2.0 ** -33, "f32": 2.0 ** -38}.get(kind[0], 0.0) * w
    half = 2.0 ** -8 if kind[1] == torch.bfloat16 else 2.0 ** -24
    # (a score of `power` bits, rounded a few times to 24: the weights move by power 2^-22 of themselves)
    rel = WEIGHT[kind[0]] + power * 2.0 ** -22 + 2.0 ** -18
    tol = want * rel + n * floor / (n + w)
    tol = tol + half * (want + tol)
    err = (out[:, 0].double().cpu() - want).abs()
    assert (err <= tol).all(), (err / tol).max().item()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 40, 1)])
def test_single_tokens_beside_chunks_as_by_themselves(tsv, kind, D, Hq, Hkv):
    """The single tokens of a mixed batch give the bits of a call of single tokens alone (the other requests bring no rows there)."""
    b = Chunk(tsv, np.random.default_rng(Hq), MIXED, Hq, Hkv, D, 16, dtype=kind[1])
    out, st = b.run(tsv, flags=kind[2])
    assert (st == 0).all()
    one = [i for i, (_, n) in enumerate(MIXED) if n == 1]
    rows = torch.from_numpy(b.offs[one]).cuda()
    b.q = b.q[rows].contiguous()
    b.offs = np.concatenate([[0], np.cumsum([int(n == 1) for _, n in MIXED])])
    alone, st = b.run(tsv, flags=kind[2], max_rows=1)
    assert (st == 0).all()
    if kind[0] == "f32":  # a kernel of its own
        assert (alone.double() - out[rows].double()).abs().max().item() <= 2.0 ** -18 * out.abs().max().item()
    else:
        assert torch.equal(alone, out[rows])


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("page,D,window", [(16, 128, 100), (16, 64, 37), (32, 64, 333)])
def test_scales_of_pages_given_away_may_be_anything(tsv, kind, page, D, window):
    """Pages in front of every window, as never written memory may have them: scales of NaN, infinity and below 0 change no bit."""
    b = Chunk(tsv, np.random.default_rng(page + D), [(1000, 70), (900, 3), (1205, 1), (507, 150)], 4, 2, D, page, dtype=kind[1])
    want, st = b.run(tsv, flags=kind[2], window=window)
    b.check(want, st, kind[2], window=window)
    front = np.concatenate([b.table[i][:max(0, p - window + 1) // page] for i, (p, _) in enumerate(b.lens)]).astype(np.int64)
    ids = torch.from_numpy(front).cuda()
    for scale in (float("nan"), float("inf"), -1.0):
        b.cache.k_scale[ids] = b.cache.v_scale[ids] = scale
        out, st = b.run(tsv, flags=kind[2], window=window)
        assert (st == 0).all() and torch.equal(out, want)
