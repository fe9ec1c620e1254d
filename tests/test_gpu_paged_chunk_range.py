"""Chunk attention and page lists on the GPU where calls meet: workspaces that kernels share, timeouts that stay reported, batches in
which requests go to two launches, verification that runs beside a call, large pools and lists whose counts do not add up."""
import numpy as np
import pytest
import torch

import _pages_ref as P
from test_gpu_paged import dev, i32, make_cache
from test_gpu_paged_chunk import KINDS, Chunk
from test_gpu_pages import Pool, lists_of

pytestmark = pytest.mark.gpu

SINGLES = [(300, 1), (0, 1), (1000, 1), (16, 1), (127, 1), (128, 1), (0, 0), (77, 1)] * 2
MIXED = SINGLES + [(40, 150), (0, 129), (500, 2)]  # enough requests, and few enough rows, for single tokens to be a launch of their own


# ------------------------------------------------------------------ attention


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 40, 1), (128, 9, 3)])
def test_single_tokens_beside_chunks(tsv, kind, D, Hq, Hkv):
    """A request's rows are right whatever else is in the batch, and a single token's the same as in a call of its own kind."""
    b = Chunk(tsv, np.random.default_rng(Hq), MIXED, Hq, Hkv, D, 16, dtype=kind[1])
    for window in (0, 100):
        out, st = b.run(tsv, flags=kind[2], window=window)
        b.check(out, st, kind[2], window=window)


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_mixed_requests_are_rejected_one_by_one(tsv, kind):
    b = Chunk(tsv, np.random.default_rng(3), MIXED, 8, 2, 128, 16, dtype=kind[1])
    good, st = b.run(tsv, flags=kind[2])
    assert (st == 0).all()
    table, start = b.table.copy(), b.start.copy()
    b.table[0][3], b.table[16][1] = -1, b.cache.num_pages  # a single token's page, a chunk's page
    b.start[2], b.start[17] = -1, 1 << 20                  # rows in front: fewer than none, more than the list holds
    out, st = b.run(tsv, flags=kind[2])
    want = [0] * len(MIXED)
    for i in (0, 16, 2, 17):
        want[i] = 1
    assert st.tolist() == want
    for i in range(len(MIXED)):
        if not want[i]:
            assert torch.equal(out[b.offs[i]:b.offs[i + 1]], good[b.offs[i]:b.offs[i + 1]])
    b.table, b.start = table, start
    # more rows than max_rows says
    _, st = b.run(tsv, flags=kind[2], max_rows=140)
    assert st.tolist() == [0] * 16 + [1, 0, 0]


def test_one_workspace_for_every_kernel(tsv):
    """Calls that differ in kernel take turns in one workspace, the size of the largest."""
    rng = np.random.default_rng(4)
    one, mixed, long = (Chunk(tsv, rng, lens, 8, 2, 128, 16) for lens in (SINGLES, MIXED, [(900, 300), (3000, 40)]))
    ws = tsv.paged_chunk_attention_workspace(mixed.q, mixed.cache, len(MIXED), mixed.max_rows)
    assert ws.numel() >= tsv.paged_chunk_attention_workspace(one.q, one.cache, 128, 1).numel()
    alone = [b.run(tsv)[0] for b in (one, mixed, long)]
    for _ in range(3):
        for b, want in zip((one, mixed, long), alone):
            out, st = b.run(tsv, workspace=ws)
            assert torch.equal(out, want) and (st == 0).all()


@pytest.mark.parametrize("lens", [[(100, 30), (0, 200)], SINGLES, MIXED], ids=["chunks", "tokens", "both"])
def test_a_chunk_timeout_is_not_overwritten(tsv, lens):
    """Words at the start of a workspace that are set stand for CTAs that gave up a wait: no call reports success over them
    until they are zero again."""
    b = Chunk(tsv, np.random.default_rng(5), lens, 8, 2, 128, 16)
    ws = tsv.paged_chunk_attention_workspace(b.q, b.cache, len(lens), b.max_rows)
    good, st = b.run(tsv, workspace=ws)
    assert (st == 0).all()
    ws.view(torch.int32)[:len(lens):2] = 1
    want = [tsv.TSV_ERR_TIMEOUT if i % 2 == 0 else 0 for i in range(len(lens))]
    for _ in range(2):
        _, st = b.run(tsv, workspace=ws)
        assert st.tolist() == want
    ws.zero_()
    out, st = b.run(tsv, workspace=ws)
    assert torch.equal(out, good) and (st == 0).all()


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: k[0])
def test_no_rows_under_a_larger_maximum(tsv, kind):
    """No rows at all, requests of none, and rows of q and out that no request has: nothing is written."""
    b = Chunk(tsv, np.random.default_rng(6), [(5, 0), (0, 0)], 4, 2, 64, 16, dtype=kind[1])
    for window in (0, 7):
        out, st = b.run(tsv, flags=kind[2], max_rows=40, window=window)
        assert out.shape == (0, 4, 64) and (st == 0).all()
    b = Chunk(tsv, np.random.default_rng(6), [(5, 40), (0, 3)], 4, 2, 64, 16, dtype=kind[1])
    want, _ = b.run(tsv, flags=kind[2])
    n = b.q.shape[0]
    q = torch.full((n + 9, 4, 64), float("nan"), dtype=b.q.dtype, device="cuda")
    q[:n] = b.q
    b.q = q
    out = torch.full_like(q, 3.0)
    out, st = b.run(tsv, flags=kind[2], out=out, max_rows=40)
    assert (st == 0).all() and torch.equal(out[:n], want) and (out[n:] == 3.0).all()


@pytest.mark.parametrize("between", ["chunk", "tokens", "both", "f32", "resize", "fork", "large fork", "compact", "large compact", "copy"])
def test_overlapped_verification_behind_a_call(tsv, between):
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
    ws = torch.zeros(tsv.tsv_tree_verify_greedy_workspace_size(tsv.handle(), B, N, V), dtype=torch.uint8, device="cuda")
    g = tsv.tree_verify_greedy(want, tokens, parent, offs, workspace=ws)
    assert (g["accept_len"] == n - 1).all()
    if between in ("chunk", "tokens", "both", "f32"):
        c = Chunk(tsv, rng, {"chunk": [(20, 30)], "tokens": SINGLES, "both": MIXED, "f32": [(20, 30)]}[between], 2, 2, 64, 16,
                  dtype=torch.float32 if between == "f32" else torch.bfloat16)
        a = (c.q, c.cache, dev(c.table), i32(c.start), i32(c.offs))
        kw = dict(max_rows=c.max_rows, out=torch.empty_like(c.q), status=i32([0] * len(c.lens)),
                  workspace=tsv.paged_chunk_attention_workspace(c.q, c.cache, len(c.lens), c.max_rows))
        call = lambda: tsv.paged_chunk_attention(*a, **kw)
    else:
        large = between.startswith("large")
        p = Pool(tsv, rng, 200000 if large else 3000, [20] * 8, 9000 if large else 40)
        rows, src = i32([320] * 8), i32([0, 1, 2, 3])
        out = dict(copy_src=i32([0] * 4), copy_dst=i32([0] * 4), status=i32([0] * 4))
        cache = make_cache(tsv, rng, 40, 16, 2, 64, True)
        done = tsv.pages_compact(p.pool, [p.d_table], [p.d_pages])
        st, one, to = i32([0] * 8), i32([0]), src + 9
        call = {
            "resize": lambda: tsv.pages_resize(p.pool, p.d_table, p.d_pages, rows, 16, status=st),
            "fork": lambda: tsv.pages_fork(p.pool, p.d_table[:4], p.d_pages[:4], src, rows[:4], p.d_table[4:], p.d_pages[4:], 16, out=out),
            "compact": lambda: tsv.pages_compact(p.pool, [p.d_table], [p.d_pages], out=done),
            "copy": lambda: tsv.pages_copy(cache, src, to, status=one),
        }[between.split()[-1]]
    for _ in range(3):
        logits.fill_(-1.0)
        logits[:, 0] = 0.0
        for r in g.values():
            r.fill_(-1)
        torch.cuda.synchronize()
        with tsv.verify_overlap(tsv.TSV_OVERLAP_GREEDY):
            tsv.rope(want.view(N, 64, 1024), zeros, freq, out=logits.view(N, 64, 1024))
            call()
            tsv.tree_verify_greedy(logits, tokens, parent, offs, workspace=ws, out=g)  # (nothing else is launched)
        torch.cuda.synchronize()
        assert torch.equal(logits, want)
        assert (g["status"] == 0).all() and (g["accept_len"] == n - 1).all()
        assert torch.equal(g["bonus"].long(), want.argmax(-1)[n - 1::n])


# ------------------------------------------------------------------ page lists


@pytest.mark.parametrize("width", [40, 9000], ids=["one-launch", "three"])
def test_fork_over_lists_that_are_counted_too_few(tsv, width):
    """Two lists with the same pages that count once: what gives a page back a second time is reported (the list is empty then, or
    unchanged when its pages were free before it was looked at), no count falls below 0, and other lists are served."""
    rng = np.random.default_rng(7)
    p = Pool(tsv, rng, 5000, [20, 30, 8, 8, 5, 5], width)
    p.d_table[3, :8] = p.d_table[2, :8]
    lost = p.table[3][:8]
    out = tsv.pages_fork(p.pool, p.d_table[:2], p.d_pages[:2], i32([0, 1, 1, -1]), i32([100, 320, 33, 0]), p.d_table[2:], p.d_pages[2:], 16)
    st, held = out["status"].tolist(), p.d_pages.tolist()
    assert set(st[:2]) <= {0, 1} and 1 in st[:2] and st[2:] == [0, 0] and held[4:] == [3, 5]
    refs = np.array(p.plain.refs)
    refs[p.table[2][:8]] -= 1
    refs[p.table[4][:5]] -= 1
    table = p.d_table.tolist()
    for b, (s, rows) in enumerate([(0, 100), (1, 320), (1, 33)]):
        if st[b]:
            assert held[2 + b] in (0, 8) and int(out["copy_dst"][b]) == -1
            continue
        full = rows // 16
        assert held[2 + b] == -(-rows // 16) and table[2 + b][:full] == p.table[s][:full]
        refs[p.table[s][:full]] += 1
        if rows % 16:
            assert int(out["copy_src"][b]) == p.table[s][full]
            refs[table[2 + b][full]] += 1
    assert p.pool.refs.tolist() == refs.tolist() and all(refs[x] == 1 for x in lost)
    assert table[:2] == lists_of(p.table[:2])


@pytest.mark.parametrize("off", [0, 1, 2, 3])
@pytest.mark.parametrize("pages", [1000, 131072, 131073, 200001])
def test_compact_into_any_alignment(tsv, pages, off):
    """Outputs that are aligned to four bytes alone; pools on both sides of where a compaction is several launches."""
    from tree_speculative_verification_attention_gb300 import pages as M

    rng = np.random.default_rng(pages + off)
    for live in (0.0, 0.4, 1.0):
        refs = (rng.random(pages) < live) * rng.integers(1, 4, size=pages)
        plain, pool = P.Pool(refs.astype(np.int32)), tsv.PagePool(i32(refs))
        space = [torch.full((pages + 8,), -5, dtype=torch.int32, device="cuda") for _ in range(4)]
        new_id, counts, src, dst = (s[off:] for s in space)
        moved = i32([-1])
        M.tsv_pages_compact(tsv.handle(), pool.c, counts.data_ptr(), None, 0, new_id.data_ptr(), src.data_ptr(), dst.data_ptr(),
                            moved.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
        want = P.compact(plain, [], [])
        m = int(moved)
        assert m == len(want[2]) and src[:m].tolist() == want[2] and dst[:m].tolist() == want[3]
        assert counts[:pages].tolist() == want[0] and new_id[:pages].tolist() == want[1]
        assert (src[m:] == -5).all() and (dst[m:] == -5).all() and (counts[pages:] == -5).all() and (new_id[pages:] == -5).all()
        for s in space:
            assert (s[:off] == -5).all()
        assert pool.refs.tolist() == refs.tolist()


@pytest.mark.parametrize("page", [16, 64])
def test_fork_at_the_border_between_one_launch_and_three(tsv, page):
    """Lists with room for 32768 entries in all, and for one more each; lists of no rows, of whole pages alone and of none."""
    rng = np.random.default_rng(8)
    for width in (4096, 4097):
        p = Pool(tsv, rng, 60000, [4000, 3000] + [int(x) for x in rng.integers(0, 2000, size=8)], width)
        src = [0, 1, 0, -1, 1, 0, 1, 1]
        rows = [4000 * page, 3000 * page - 1, 0, 0, page, page - 1, 1, 2999 * page + 1]
        out = tsv.pages_fork(p.pool, p.d_table[:2], p.d_pages[:2], i32(src), i32(rows), p.d_table[2:], p.d_pages[2:], page)
        child, has = p.table[2:], p.pages[2:]
        want = P.fork(p.plain, p.table[:2], p.pages[:2], src, rows, child, has, page)
        p.table[2:], p.pages[2:] = child, has
        assert [out[x].tolist() for x in ("copy_src", "copy_dst", "status")] == list(want)
        p.same()


def test_lists_shared_by_two_streams_and_two_graphs(tsv):
    """Calls on pools of their own, captured into two graphs that run at once: nothing is shared behind their backs."""
    rng = np.random.default_rng(9)
    ps = [Pool(tsv, rng, n, [300] * 20, 500) for n in (20000, 160000)]
    graphs, rows, outs = [], [], []
    for p in ps:
        r, st, s = i32([0] * 20), i32([0] * 20), torch.cuda.Stream()
        done = tsv.pages_compact(p.pool, [p.d_table], [p.d_pages])
        before = [x.clone() for x in (p.pool.refs, p.d_table, p.d_pages)]
        graph = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            tsv.pages_resize(p.pool, p.d_table, p.d_pages, r, 16, status=st)
            tsv.pages_compact(p.pool, [p.d_table], [p.d_pages], out=done)
        for x, was in zip((p.pool.refs, p.d_table, p.d_pages), before):
            assert torch.equal(x, was)
        graphs.append((graph, s)), rows.append(r), outs.append((st, done))
    for _ in range(4):
        want = []
        for p, r in zip(ps, rows):
            w = [int(x) for x in rng.integers(0, 500 * 16 + 1, size=20)]
            r.copy_(i32(w))
            want.append((P.resize(p.plain, p.table, p.pages, w, 16), P.compact(p.plain, [p.table], [p.pages])))
        torch.cuda.synchronize()
        for graph, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for p, (st, done), (w, moved) in zip(ps, outs, want):
            assert st.tolist() == w
            p.same()
            assert done["refs"].tolist() == moved[0] and done["new_id"].tolist() == moved[1] and int(done["moved"]) == len(moved[2])


def test_copies_of_many_pages_and_few_of_them(tsv):
    """Room for far more pairs than the count on the device says, in a grid that is not as large as the units."""
    rng = np.random.default_rng(10)
    c = make_cache(tsv, rng, 3000, 16, 2, 64, True)
    k, v, ks, vs = (x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale))
    ids = rng.permutation(3000)
    src, dst = np.full(60000, -1), np.full(60000, -1)
    src[:1400], dst[:1400] = ids[:1400], ids[1500:2900]
    for n in (1400, 7, 0, 60000):
        for now, was in ((c.k, k), (c.v, v), (c.k_scale, ks), (c.v_scale, vs)):
            now.copy_(was)
        st = tsv.pages_copy(c, i32(src), i32(dst), count=i32([n]))
        assert st.tolist() == [0]
        m = min(n, 1400)
        s, d = torch.tensor(src[:m]).cuda(), torch.tensor(dst[:m]).cuda()
        for now, was in ((c.k, k), (c.v, v), (c.k_scale, ks), (c.v_scale, vs)):
            now, want = now.view(torch.uint8), was.clone().view(torch.uint8)
            want[d] = want[s]
            assert torch.equal(now, want)
