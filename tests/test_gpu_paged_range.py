"""Ranges of the paged 8-bit cache's operators on the GPU: scales far from one another, the smallest and largest ones, full
batches.  Against the 64-bit forms of tests/_paged_ref.py under the bounds of test_gpu_paged.py."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import _paged_ref as R
from test_gpu_paged import KINDS, Batch, _attention_bound, accepted, dev, i32, same_codes, values, wide_workspace

pytestmark = pytest.mark.gpu

LENS = [(37, 5), (300, 3), (0, 8), (256, 1), (700, 4)]  # prefix, nodes (8 at most)
ROWS = [(16, 4, 2), (32, 8, 2), (64, 64, 8)]  # query rows a unit, Hq, Hkv: 8 nodes times Hq / Hkv


def run_of(tsv, b, rows, flags=0):
    """The call that takes units of so many rows (256: the kernel of many rows)."""
    return b.run(tsv, flags=flags, workspace=wide_workspace(tsv, b) if rows == 256 else None)


# ------------------------------------------------------------------ values of zero


def zero_values(b, where, head=0):
    """V of one head zero in some of the pages, under the scale that append and commit write for zeros."""
    pages = []
    for i, (p, n) in enumerate(b.lens):
        main = b.table[i][:-(-p // b.page)].tolist()
        tree = b.tree_table[i][:-(-n // b.page)].tolist()
        front = 256 // b.page
        pages += {"all": main + tree, "front": main[:front], "back": main[front:] + tree, "tree": tree}[where]
    ids = torch.tensor(pages, device="cuda")
    b.cache.v.view(torch.uint8)[ids, :, head] = 0
    b.cache.v_scale[ids, head] = 2.0 ** -126


ZERO = ["all", "front", "back", "tree"]


@pytest.mark.parametrize("where", ZERO)
@pytest.mark.parametrize("page,D", [(16, 128), (64, 64)])
@pytest.mark.parametrize("rows,Hq,Hkv", ROWS)
def test_zero_values(tsv, rows, Hq, Hkv, page, D, where):
    """Weights times zeros are zeros, whatever is masked, and ordinary values beside them are as exact as alone."""
    b = Batch(tsv, np.random.default_rng(101), LENS, Hq, Hkv, D, page)
    zero_values(b, where)
    out, st = run_of(tsv, b, rows)
    b.check(out, st, True)
    if where == "all":
        assert (out[:, :Hq // Hkv] == 0).all()


@pytest.mark.parametrize("where", ZERO)
@pytest.mark.parametrize("long", [0, 6000])
@pytest.mark.parametrize("page,D", [(16, 128), (64, 64)])
def test_zero_values_of_many_rows(tsv, page, D, long, where):
    """The same in units of 256 rows, whole and cut."""
    lens = [(p + long * (i == 1), n) for i, (p, n) in enumerate(LENS)]
    b = Batch(tsv, np.random.default_rng(102), lens, 256, 8, D, page)
    zero_values(b, where)
    out, st = run_of(tsv, b, 256)
    b.check(out, st, True)
    if where == "all":
        assert (out[:, :32] == 0).all()


@pytest.mark.parametrize("rows", [0, 16, 32, 64, 256])
def test_zero_values_written_by_append(tsv, rows):
    """A KV head whose V is zero throughout, prefix and tree written by append (rows 0: on CUDA cores)."""
    Hq, Hkv = {0: (4, 2), 16: (4, 2), 32: (8, 2), 64: (64, 8), 256: (256, 8)}[rows]
    rng = np.random.default_rng(103)
    b = Batch(tsv, rng, LENS, Hq, Hkv, 128, 32)
    for table, sizes in ((b.table, [p for p, _ in LENS]), (b.tree_table, [n for _, n in LENS])):
        offs = np.concatenate([[0], np.cumsum(sizes)])
        k, v = (dev(rng.normal(size=(int(offs[-1]), Hkv, 128)), torch.bfloat16) for _ in range(2))
        v[:, 1] = 0
        assert (tsv.paged_append(b.cache, dev(table), k, v, i32(offs)) == 0).all()
    out, st = run_of(tsv, b, rows, flags=1 if rows == 0 else 0)
    b.check(out, st, rows > 0)
    G = Hq // Hkv
    assert (out[:, G:2 * G] == 0).all()


@pytest.mark.parametrize("rows", [0, 16, 32, 64, 256])
@pytest.mark.parametrize("power", [-126, -120, -110, 100, 127])
def test_a_scale_is_a_factor(tsv, rows, power):
    """V scales of 2^power give 2^power times what scales of one give, from the smallest to the largest fp32 holds (2^127:
    with values of 2^-6 at most).  Powers of two change no rounding, but results below 2^-126 have bf16's step of 2^-133,
    and products of weights and scales below it fp32's of 2^-149, which is 2^-23 of the largest."""
    Hq, Hkv = {0: (4, 2), 16: (4, 2), 32: (8, 2), 64: (64, 8), 256: (256, 8)}[rows]
    b = Batch(tsv, np.random.default_rng(104), LENS, Hq, Hkv, 128, 16)
    if power == 127:
        v = b.cache.v.view(torch.uint8)
        v.copy_((v & 0x80) | (v & 0x07))
    flags = 1 if rows == 0 else 0
    b.cache.v_scale.fill_(1.0)
    one = run_of(tsv, b, rows, flags)[0].double()
    b.cache.v_scale.fill_(2.0 ** power)
    out, st = run_of(tsv, b, rows, flags)
    assert (st == 0).all() and torch.isfinite(out).all()
    err = (out.double() * 2.0 ** -power - one).abs()
    if power >= -110:  # (results of 2^-126 and more are one of 2^-16, of which none here is less but zeros)
        assert (err <= 2.0 ** (-133 - power)).all()
    else:
        # one bf16 step where 2^-21 moves a value over the border between two
        top = b.cache.v.float().abs().amax().item()
        assert (err <= 2.0 ** -7 * one.abs() + 2.0 ** -20 * top + 2.0 ** (-133 - power)).all()


# ------------------------------------------------------------------ V scales far apart


def lost(b, floor):
    """How far outputs may be off beyond _attention_bound because a weight (p times its V scale) is off by at most `floor` of
    its row's largest, or, next to nothing, lost: the sums of min(weight, floor x largest) |code| [N, Hq, D]."""
    c, G = values(b.cache), b.Hq // b.Hkv
    out = np.zeros((len(b.q), b.Hq, b.D))
    q = b.q.double().cpu().numpy()
    for r, (P, n) in enumerate(b.lens):
        ids = np.concatenate([b.table[r][np.arange(P) // b.page], b.tree_table[r][np.arange(n) // b.page]])
        rows = np.concatenate([np.arange(P), np.arange(n)]) % b.page
        k, codes = c.k[ids, rows] * c.k_scale[ids][:, :, None], np.abs(c.v[ids, rows])
        for i in range(n):
            see = np.concatenate([np.ones(P, bool), b.sees[b.offs[r] + i, :n]])
            for h in range(b.Hq):
                s = k[see, h // G] @ q[b.offs[r] + i, h] / math.sqrt(b.D)
                p = np.exp(s - s.max())
                w = p / p.sum() * c.v_scale[ids[see], h // G]
                out[b.offs[r] + i, h] = np.minimum(w, floor * w.max()) @ codes[see, h // G]
    return out


@pytest.mark.parametrize("rows", [0, 16, 32, 64, 256])
@pytest.mark.parametrize("page,D", [(16, 128), (128, 64), (32, 128)])
def test_pages_whose_values_lie_far_apart(tsv, rows, page, D):
    """V scales 2^30 apart from page to page and rows that attend to hardly more than one key: the weights of a page of
    small values are held as well as those of a page of large ones beside it."""
    Hq, Hkv = {0: (4, 2), 16: (4, 2), 32: (8, 2), 64: (64, 8), 256: (256, 8)}[rows]
    rng = np.random.default_rng(105)
    lens = [(p + 256 * i, n) for i, (p, n) in enumerate(LENS)]
    b = Batch(tsv, rng, lens, Hq, Hkv, D, page)
    pages = torch.arange(b.cache.num_pages, device="cuda")
    b.cache.v_scale.mul_((2.0 ** ((pages * 7) % 31 - 30.0)).unsqueeze(1))
    b.q[::2] *= 60.0  # rows of one key, and flat ones
    out, st = run_of(tsv, b, rows, flags=1 if rows == 0 else 0)
    assert (st == 0).all()
    ref, spread, size = R.attention(b.q.double().cpu().numpy(), values(b.cache), b.table, b.prefix, b.offs, b.tree_table, b.sees)
    tol = _attention_bound(ref, spread, size, b.q.dtype, max(p + n for p, n in lens), D, rows > 0)
    # Few rows: a weight is two e4m3 terms whose smallest step is 2^-9, the second off by half of it: 2^-10, of 256 for the
    # step's largest p times scale, or of 2^4 less where the step's scales are no further apart than that: 2^-14 of the row's
    # largest at most.  Many rows: fp16 of 2^11 or more for the largest, off by 2^-25: 2^-36.  The reference takes p times the
    # scale in fp32, whose own rounding _attention_bound has.
    if rows > 0:
        tol += lost(b, 2.0 ** -36 if rows == 256 else 2.0 ** -14) * (1 + 2.0 ** -7)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), ((err / tol).max(), np.argwhere(err > tol)[:4])
    # the rows of one key do reach pages of small values
    assert (np.abs(ref).max(axis=-1) < 2.0 ** -12 * np.abs(ref).max()).any()


# ------------------------------------------------------------------ workspaces


@pytest.mark.parametrize("rows", [16, 32, 64, 256])
def test_a_timeout_is_not_overwritten(tsv, rows):
    """Words of a workspace that are set stand for CTAs that gave up a wait before the requests were checked: the checks do
    not report success over them, in this call or a later one.  Zeroed again, the workspace is as good as new."""
    Hq, Hkv = {16: (4, 2), 32: (8, 2), 64: (64, 8), 256: (256, 8)}[rows]
    b = Batch(tsv, np.random.default_rng(106), LENS, Hq, Hkv, 128, 16)
    if rows == 256:
        wide_workspace(tsv, b)
    ws = tsv.paged_tree_attention_workspace(b.q, b.cache, len(LENS), 8)
    good, st = b.run(tsv, workspace=ws)
    assert (st == 0).all()
    ws.fill_(1)
    for _ in range(2):
        _, st = b.run(tsv, workspace=ws)
        assert (st == tsv.TSV_ERR_TIMEOUT).all()
    ws.zero_()
    out, st = b.run(tsv, workspace=ws)
    assert torch.equal(out, good) and (st == 0).all()


# ------------------------------------------------------------------ order of launches


@pytest.mark.parametrize("between", ["rope", "append", "attention", "commit"])
def test_overlapped_verification_behind_a_paged_call(tsv, between):
    """A verification that may run beside the call before it still comes behind the one before that: here a rotation by 0 that
    writes its logits in one long wave of blocks."""
    rng = np.random.default_rng(107)
    B, n, V = 19, 128, 65536
    N = B * n
    want = torch.randn(N, V, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    logits = torch.empty_like(want)
    parent = i32(np.tile(np.arange(-1, n - 1), B))
    offs = i32(np.arange(B + 1) * n)
    tokens = torch.cat([want[:1].argmax(-1), want.argmax(-1)[:-1]]).int()  # every node accepted
    zeros, freq = i32(np.zeros(N)), tsv.rope_frequencies(1024, device="cuda")[0]
    b = Batch(tsv, rng, [(20, 3)], 2, 2, 64, 16, spare=4)
    kv = b.q.clone()
    small = tsv.rope_frequencies(64, device="cuda")[0]
    ws = torch.zeros(tsv.tsv_tree_verify_greedy_workspace_size(tsv.handle(), B, N, V), dtype=torch.uint8, device="cuda")
    g = tsv.tree_verify_greedy(want, tokens, parent, offs, workspace=ws)
    assert (g["accept_len"] == n - 1).all()
    d = dict(table=dev(b.table), tree=dev(b.tree_table), plen=i32(b.prefix), offs=i32(b.offs), anc=dev(b.words), path=i32([0, 1, 2]), last=i32([2]))
    out, st = torch.empty_like(b.q), torch.empty(1, dtype=torch.int32, device="cuda")
    res = dict(new_len=torch.empty_like(st), status=torch.empty_like(st))
    calls = {
        "rope": lambda: tsv.rope(kv, d["path"], small, out=out),
        "append": lambda: tsv.paged_append(b.cache, d["tree"], kv, kv, d["offs"], status=st),
        "attention": lambda: tsv.paged_tree_attention(b.q, b.cache, d["table"], d["plen"], d["offs"], tree_table=d["tree"], anc=d["anc"],
                                                      max_nodes=3, flags=1, out=out, status=st),
        "commit": lambda: tsv.paged_commit(b.cache, d["table"], d["tree"], d["plen"], d["offs"], d["path"], d["last"], out=res),
    }
    for _ in range(3):
        logits.fill_(-1.0)
        logits[:, 0] = 0.0
        for r in g.values():
            r.fill_(-1)
        torch.cuda.synchronize()
        with tsv.verify_overlap(tsv.TSV_OVERLAP_GREEDY):
            tsv.rope(want.view(N, 64, 1024), zeros, freq, out=logits.view(N, 64, 1024))
            calls[between]()
            tsv.tree_verify_greedy(logits, tokens, parent, offs, workspace=ws, out=g)  # (nothing else is launched)
        torch.cuda.synchronize()
        assert torch.equal(logits, want)
        assert (g["status"] == 0).all() and (g["accept_len"] == n - 1).all()
        assert torch.equal(g["bonus"].long(), want.argmax(-1)[n - 1::n])


# ------------------------------------------------------------------ angles


def test_rope_angles_to_the_last_bit(tsv):
    """Pairs (1, 0) turn into (cosine, sine) of the angle.  A frequency is kept to half of 2^-64 turns, and nothing of its
    product with the position is dropped: the angle is off by |position| 2^-65 turns.  Then cosine and sine of its upper part
    (2^-22 of each), turned on by the rest r of at most 64 x 2^-32 turns: 2^-22 more for the rounding, r^2 / 2 < 2^-47 for the
    second order, and 2^-22 r < 2^-45 where sine and rest cancel."""
    two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889")
    steps = [k + f for k in (0, 1, 2, 3, 63, 64, 65, 127, 128, 1000) for f in (0.5, 0.9, 0.99)]
    w = [2 * math.pi * s / 2 ** 32 for s in steps] + [2 * math.pi * s / 2 ** 64 for s in steps]
    w += [math.pi - x for x in w[:30]] + [math.pi * (1 - 2.0 ** -k) for k in range(2, 40)] + [10000.0 ** (-i / 64) for i in range(64)]
    half = len(w)
    pos = [1, -1, 3, 1 << 20, 2 ** 31 - 1, -2 ** 31]
    x = torch.zeros(len(pos), 1, 2 * half, device="cuda")
    x[..., :half] = 1.0
    got = tsv.rope(x, i32(pos), torch.tensor(w, dtype=torch.float64, device="cuda")).double().cpu().numpy()[:, 0]
    for n, p in enumerate(pos):
        for i, f in enumerate(w):
            t = Fraction(f) * p / two_pi
            t = float((t - round(t)) * two_pi)
            for have, ref in ((got[n, i], math.cos(t)), (got[n, half + i], math.sin(t))):
                tol = 2.0 ** -21 * abs(ref) + 2.0 ** -44 + 2 * math.pi * abs(p) * 2.0 ** -65
                assert abs(have - ref) <= tol, (p, f, have, ref, abs(have - ref) / tol)


def test_commit_rejects_the_largest_accept_len(tsv):
    """accept_len + 1 does not overflow."""
    b = Batch(tsv, np.random.default_rng(108), [(5, 3), (7, 4)], 2, 2, 64, 16)
    before = values(b.cache)
    for big in (2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31):
        o = tsv.paged_commit(b.cache, dev(b.table), dev(b.tree_table), i32(b.prefix), i32(b.offs), i32([0, 1, 2, 0, 1, 2, 3]),
                             i32([big, big]))
        assert o["status"].tolist() == [1, 1] and o["new_len"].tolist() == [-1, -1]
    same_codes(b.cache, before)


# ------------------------------------------------------------------ full batches


@pytest.mark.parametrize("rows", [0, 16, 32, 64, 256])
def test_full_batches_through_a_step(tsv, rows):
    """128 requests, where the lists of a call are full: attention, the commit of a path whose rows end in the next page (the
    cache against the 64-bit form), and attention over the longer prefixes."""
    Hq, Hkv, most = {0: (4, 2, 8), 16: (4, 2, 8), 32: (8, 2, 8), 64: (32, 4, 8), 256: (64, 2, 8)}[rows]
    rng = np.random.default_rng(109)
    lens = [(int(rng.integers(0, 300)), int(rng.integers(1, most + 1))) for _ in range(128)]
    lens[5] = (15, most)
    b = Batch(tsv, rng, lens, Hq, Hkv, 64, 16, spare=130)
    kw = dict(flags=1 if rows == 0 else 0)
    if rows == 256:
        kw["workspace"] = wide_workspace(tsv, b)
    out, st = b.run(tsv, **kw)
    b.check(out, st, rows > 0)
    used = set(b.table[b.table >= 0]) | set(b.tree_table[b.tree_table >= 0])
    free = [i for i in range(b.cache.num_pages) if i not in used]
    path, acc, ref = np.full(int(b.offs[-1]), -1), [], values(b.cache)
    b.table = np.concatenate([b.table, np.full((128, 1), -1, dtype=np.int32)], axis=1)
    for i, (p, n) in enumerate(lens):
        way = accepted(rng, b.parent[b.offs[i]:b.offs[i] + n], n)
        path[b.offs[i]:b.offs[i] + len(way)] = way
        acc.append(len(way) - 1)
        if -(-(p + len(way)) // 16) > -(-p // 16):
            b.table[i, -(-p // 16)] = free.pop()
        k, v = ref.rows(b.tree_table[i], n)
        ref.write(b.table[i], p, k[way], v[way])
    o = tsv.paged_commit(b.cache, dev(b.table), dev(b.tree_table), i32(b.prefix), i32(b.offs), i32(path), i32(acc))
    assert (o["status"] == 0).all()
    same_codes(b.cache, ref)
    b.lens = [(p + a + 1, n) for (p, n), a in zip(lens, acc)]
    b.prefix = np.array([p for p, _ in b.lens])
    assert o["new_len"].tolist() == b.prefix.tolist()
    out, st = b.run(tsv, **kw)
    b.check(out, st, rows > 0)


# ------------------------------------------------------------------ captured steps


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_a_captured_step_gives_what_eager_calls_give(tsv, kind):
    """Rotation, append, attention and commit in one graph, replayed with other positions, lengths and paths on the device:
    results and cache bit for bit as from single calls, those on a stream of their own too."""
    rng = np.random.default_rng(110)
    dtype, flags = kind[1], kind[2]
    b = Batch(tsv, rng, [(100, 9), (31, 3), (0, 6)], 8, 2, 128, 16, dtype=dtype, spare=20)
    N, B = len(b.q), 3
    used = set(b.table[b.table >= 0]) | set(b.tree_table[b.tree_table >= 0])
    free = [i for i in range(b.cache.num_pages) if i not in used]
    table = np.concatenate([b.table, np.full((B, 2), -1, dtype=np.int32)], axis=1)
    for i in range(B):
        for x in range(table.shape[1]):
            if table[i, x] < 0 and free:
                table[i, x] = free.pop()
    freq = tsv.rope_frequencies(128, device="cuda")[0]
    d = dict(table=dev(table), tree=dev(b.tree_table), plen=i32(b.prefix), offs=i32(b.offs), anc=dev(b.words), pos=i32(np.zeros(N)),
             path=i32(np.full(N, -1)), acc=i32(np.zeros(B)))
    kv = dev(rng.normal(size=(N, 2, 2, 128)), dtype)
    start = [t.clone() for t in (b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8), b.cache.k_scale, b.cache.v_scale)]

    def restore():
        for to, was in zip((b.cache.k.view(torch.uint8), b.cache.v.view(torch.uint8), b.cache.k_scale, b.cache.v_scale), start):
            to.copy_(was)

    def buffers():
        return dict(q=torch.empty_like(b.q), out=torch.full_like(b.q, 7.0), s1=i32([7] * B), s2=i32([7] * B),
                    res=dict(new_len=i32([7] * B), status=i32([7] * B)),
                    ws=tsv.paged_tree_attention_workspace(b.q, b.cache, B, 9, flags=flags))

    def step(o, stream=None):
        tsv.rope(b.q, d["pos"], freq, out=o["q"], stream=stream)
        tsv.paged_append(b.cache, d["tree"], kv[:, 0], kv[:, 1], d["offs"], positions=d["pos"], inv_freq=freq, status=o["s1"], stream=stream)
        tsv.paged_tree_attention(o["q"], b.cache, d["table"], d["plen"], d["offs"], tree_table=d["tree"], anc=d["anc"], max_nodes=9,
                                 flags=flags, out=o["out"], workspace=o["ws"], status=o["s2"], stream=stream)
        tsv.paged_commit(b.cache, d["table"], d["tree"], d["plen"], d["offs"], d["path"], d["acc"], max_nodes=9, out=o["res"], stream=stream)

    def results(o):
        torch.cuda.synchronize()
        c = b.cache
        return [t.clone() for t in (o["q"], o["out"], o["s1"], o["s2"], o["res"]["new_len"], o["res"]["status"],
                                    c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]

    o, graph, side = buffers(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    step(o)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(o)
    for lens in ([100, 31, 0], [17, 0, 5], [64, 16, 1], [3, -1, 2]):
        path, acc = np.full(N, -1), []
        for i in range(B):
            lo, hi = b.offs[i], b.offs[i + 1]
            way = accepted(rng, b.parent[lo:hi], hi - lo)
            path[lo:lo + len(way)] = way
            acc.append(len(way) - 1)
        for name, x in (("plen", lens), ("path", path), ("acc", acc), ("pos", rng.integers(0, 5000, N))):
            d[name].copy_(i32(x))
        restore()
        o["out"].fill_(7.0)  # (the rows of a rejected request stay)
        graph.replay()
        got = results(o)
        restore()
        e = buffers()
        step(e)
        for n, (x, y) in enumerate(zip(got, results(e))):
            assert torch.equal(x, y), (lens, n)
        restore()
        e = buffers()
        side.wait_stream(torch.cuda.current_stream())
        step(e, side)
        for n, (x, y) in enumerate(zip(got, results(e))):
            assert torch.equal(x, y), (lens, n)
        assert got[3].tolist() == got[5].tolist() == [1 if p < 0 else 0 for p in lens]
