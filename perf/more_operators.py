"""Cases of the operators around a paged 8-bit KV cache that a serving loop needs beside its tree attention, and their plain forms.

Five operators: `attention` (a chunk of new tokens, or single ones, over the pages they were appended to), `resize` (page lists
grow and shrink against a pool with reference counts), `fork` (page lists that share another's pages), `compact` (live pages
to the low ids) and `copy` (codes and scales of pages inside a layer's cache).

The cache: pages of `page` rows, one fp32 power-of-two scale per page and KV head for K and for V; a value is code x scale.
A pool: refs[p] page lists hold page p; 0 is a free page.

`run` computes an operator in elementary torch operations in 32 bits, or, with `own` set, calls the framework.  `exact` gives the
same outputs from the definition, in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
OK, NO_PAGES = 0, 7


# ------------------------------------------------------------------ cases


def listed():
    return [
        # The first chunk of one prompt, 32 query / 8 KV heads: what a new request waits for (latency counts).
        dict(name="attn-first512-gqa32x8", op="attention", B=1, ones=0, n_lo=512, n_hi=512, p_lo=0, p_hi=0, Hq=32, Hkv=8, D=128,
             page=16, window=0, dtype="bf16", head_major=True),
        # A chunk of a long prompt, 4096 tokens behind 28672: the products are what counts.
        dict(name="attn-chunk4096-P28672-gqa64x8", op="attention", B=1, ones=0, n_lo=4096, n_hi=4096, p_lo=28672, p_hi=28672, Hq=64,
             Hkv=8, D=128, page=64, window=0, dtype="bf16", head_major=True),
        # A serving batch: 28 requests decode one token each, 4 others bring prompt chunks of different lengths.
        dict(name="attn-mixed32-gqa32x8", op="attention", B=32, ones=28, n_lo=100, n_hi=1000, p_lo=0, p_hi=8000, Hq=32, Hkv=8, D=128,
             page=32, window=0, dtype="bf16", head_major=True),
        # Ragged chunks in fp32 under a sliding window, heads of 64, token-major pages.
        dict(name="attn-ragged-f32-window500", op="attention", B=5, ones=1, n_lo=1, n_hi=700, p_lo=0, p_hi=1500, Hq=8, Hkv=2, D=64,
             page=16, window=500, dtype="f32", head_major=False),
        # Tree pages for one speculation step of 32 requests, taken and given back.
        dict(name="resize-tree32", op="resize", B=32, pool=8192, page=16, held_lo=10, held_hi=150, more_lo=1, more_hi=4, spare=2.0),
        # Room for the prompts of 128 requests in a large pool in use for long, taken and given back.
        dict(name="resize-prompts128", op="resize", B=128, pool=1 << 20, page=16, held_lo=0, held_hi=4096, more_lo=0, more_hi=2048,
             spare=1.2),
        # Eight samples continue one prompt of 1100 tokens.
        dict(name="fork-sample8", op="fork", B=8, parents=1, pool=4096, page=16, rows_lo=1100, rows_hi=1100),
        # 128 beams take over the lists of 16 others, 8192 to 32768 tokens each.
        dict(name="fork-beam128", op="fork", B=128, parents=16, pool=1 << 17, page=16, rows_lo=8192, rows_hi=32768),
        # A small pool, half in use.
        dict(name="compact-4096", op="compact", B=16, pool=4096, held_lo=64, held_hi=192, shared=0.1),
        # A pool of a million pages, 128 lists of up to 8192 pages.
        dict(name="compact-1M", op="compact", B=128, pool=1 << 20, held_lo=2000, held_hi=8192, shared=0.2),
        # The last pages of eight forks.
        dict(name="copy-fork8", op="copy", n=8, pool=4096, Hkv=8, D=128, page=16, layout="head"),
        # What a compaction moves in one layer: 4096 pages of 64 tokens, 0.5 GB.
        dict(name="copy-compact4096", op="copy", n=4096, pool=8300, Hkv=8, D=128, page=64, layout="head"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "resize", "fork", "compact", "copy"])
    if op == "attention":
        f32 = rng.random() < 0.2
        Hkv, G = rng.choice([1, 2, 3, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8])
        kind = rng.choice(["chunks", "mixed", "tokens"])
        B = _log_int(rng, 1, 6 if f32 else 32)
        ones = B if kind == "tokens" else rng.randint(0, B - 1) if kind == "mixed" else 0
        # rows of q: the products of the largest listed case and its keys are not passed
        n_hi = _log_int(rng, 2, max(2, (2000 if f32 else 8000) // max(1, B - ones)))
        p_hi = _log_int(rng, 16, 1500 if f32 else max(16, min(28672, (1 << 18) // B)))
        return dict(op=op, B=B, ones=ones, n_lo=rng.choice([1, n_hi // 2 + 1, n_hi]), n_hi=n_hi, p_lo=rng.choice([0, p_hi // 4, p_hi]),
                    p_hi=p_hi, Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                    window=rng.choice([0, 0, _log_int(rng, 1, 4000)]), dtype="f32" if f32 else "bf16", head_major=rng.random() < 0.7)
    B = _log_int(rng, 1, 128)
    if op == "resize":
        held_hi, more_hi = _log_int(rng, 1, 4096), _log_int(rng, 1, 2048)
        low = B * (held_hi + more_hi) + 64
        return dict(op=op, B=B, pool=_log_int(rng, low, max(low, 1 << 20)), page=rng.choice([16, 32, 64, 128]), held_lo=0,
                    held_hi=held_hi, more_lo=rng.randint(0, 1), more_hi=more_hi, spare=rng.choice([0.5, 1.0, 1.2, 3.0]))
    if op == "fork":
        page, parents = rng.choice([16, 32, 64, 128]), _log_int(rng, 1, 16)
        rows_hi = _log_int(rng, 1, 32768)
        low = parents * (rows_hi // page + 2) + 2 * B + 64
        return dict(op=op, B=B, parents=parents, pool=_log_int(rng, low, max(low, 1 << 17)), page=page,
                    rows_lo=rng.choice([1, rows_hi]), rows_hi=rows_hi)
    if op == "compact":
        held_hi = _log_int(rng, 1, 8000)
        low = B * held_hi + 64
        return dict(op=op, B=B, pool=_log_int(rng, low, max(low, 1 << 20)), held_lo=0, held_hi=held_hi, shared=rng.choice([0.0, 0.3]))
    Hkv, D, page = rng.choice([1, 2, 3, 5, 8, 32]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    n = _log_int(rng, 1, (1 << 29) // (2 * page * Hkv * D))
    return dict(op=op, n=n, pool=2 * n + rng.randint(1, 100), Hkv=Hkv, D=D, page=page, layout=rng.choice(["head", "token", "fused"]))


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "attention":
        n, start = _lengths(case)
        keys, seen, w = 0, 0, case["window"]
        for nb, p in zip(n.tolist(), start.tolist()):
            if not nb:
                continue
            keys += p + nb if not w else min(p + nb, nb + w - 1)
            pos = np.arange(p, p + nb, dtype=np.int64) + 1
            seen += int((np.minimum(pos, w) if w else pos).sum())
        esz = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * keys * case["Hkv"] * case["D"] + 2 * int(n.sum()) * case["Hq"] * case["D"] * esz,
                "flops": 4 * seen * case["Hq"] * case["D"]}
    if op == "copy":
        return {"bytes": 2 * case["n"] * (2 * case["page"] * case["Hkv"] * case["D"] + 8 * case["Hkv"]) + 8 * case["n"],
                "flops": 2 * case["n"] * case["Hkv"]}
    lay = _lists(case, 0)
    if op == "resize":
        want = -(-lay["rows_up"].astype(np.int64) // case["page"])
        need = np.cumsum(np.maximum(want - lay["held"], 0))
        free = int((lay["refs"] == 0).sum())
        got = int(need[need <= free].max()) if (need <= free).any() else 0
        # the counts once to find the free pages; an entry and a count written when a page is taken, both read and the count
        # written when it is given back
        return {"bytes": 4 * case["pool"] + 20 * got, "flops": case["pool"] + 2 * got}
    if op == "fork":
        full, part = lay["rows"] // case["page"], lay["rows"] % case["page"] > 0
        old, shared = int((full + part).sum()), int(full.sum())  # (lists of the last pass, lists of this one)
        return {"bytes": 12 * old + 16 * shared + 16 * int(part.sum()), "flops": old + shared}
    moved = int((np.nonzero(lay["refs"])[0] >= (lay["refs"] > 0).sum()).sum())
    entries = int(lay["held"].sum())
    return {"bytes": 12 * case["pool"] + 8 * moved + 8 * entries, "flops": 2 * case["pool"] + entries}


# ------------------------------------------------------------------ inputs


def _put(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _lengths(case):
    """New tokens and rows in front of them, per request (they belong to the case)."""
    rng = np.random.default_rng([3, case["B"], case["n_hi"], case["p_hi"], case["ones"]])
    n = rng.integers(case["n_lo"], case["n_hi"] + 1, size=case["B"])
    n[rng.permutation(case["B"])[:case["ones"]]] = 1
    return n.astype(np.int64), rng.integers(case["p_lo"], case["p_hi"] + 1, size=case["B"]).astype(np.int64)


def _lists(case, seed):
    """Page lists and reference counts of a pool in use (host side, all from the seed; lengths belong to the case)."""
    op, B, pool = case["op"], case["B"], case["pool"]
    own_rng = np.random.default_rng([5, B, pool])
    ids = np.random.default_rng([int(seed), 11]).permutation(pool).astype(np.int32)  # a pool in use for long: no order is left
    if op == "resize":
        page = case["page"]
        held = own_rng.integers(case["held_lo"], case["held_hi"] + 1, size=B)
        more = own_rng.integers(case["more_lo"], case["more_hi"] + 1, size=B)
        rows = np.maximum(held * page - own_rng.integers(0, page, size=B), 0)
        up = np.maximum((held + more) * page - own_rng.integers(0, page, size=B), rows)
        refs = np.zeros(pool, dtype=np.int32)
        table = np.full((B, max(1, int((held + more).max()))), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            table[b, :held[b]] = ids[at:at + held[b]]
            at += int(held[b])
        free = min(pool - at, int(more.sum() * case["spare"]) + 1)
        refs[ids[:pool - free]] = 1  # (the others belong to requests of other batches)
        return dict(refs=refs, table=table, held=held.astype(np.int32), rows=rows.astype(np.int32), rows_up=up.astype(np.int32))
    if op == "fork":
        page, F = case["page"], case["parents"]
        have = own_rng.integers(case["rows_lo"], case["rows_hi"] + 1, size=F)
        held = -(-have // page)
        source = own_rng.integers(0, F, size=B)
        rows = have[source]
        refs = np.zeros(pool, dtype=np.int32)
        parents = np.full((F, int(held.max())), -1, dtype=np.int32)
        at = 0
        for f in range(F):
            parents[f, :held[f]] = ids[at:at + held[f]]
            refs[ids[at:at + held[f]]] = 1
            at += int(held[f])
        # what the children hold so far: an earlier fork, of any parent
        old = own_rng.integers(0, F, size=B)
        table = np.full((B, int(held.max())), -1, dtype=np.int32)
        for b in range(B):
            m = int(held[old[b]])
            table[b, :m - 1] = parents[old[b], :m - 1]
            np.add.at(refs, table[b, :m - 1], 1)
            table[b, m - 1] = ids[at]
            refs[ids[at]] = 1
            at += 1
        return dict(refs=refs, parents=parents, parent_pages=held.astype(np.int32), table=table, held=held[old].astype(np.int32),
                    source=source.astype(np.int32), rows=rows.astype(np.int32))
    held = own_rng.integers(case["held_lo"], case["held_hi"] + 1, size=B)
    table = np.full((B, max(1, int(held.max()))), -1, dtype=np.int32)
    refs = np.zeros(pool, dtype=np.int32)
    at = 0
    for b in range(B):
        m = int(held[b])
        share = 0
        if b and case["shared"]:  # the first pages are those of the request before
            share = min(int(held[b - 1] * case["shared"]), m)
            table[b, :share] = table[b - 1, :share]
        table[b, share:m] = ids[at:at + m - share]
        at += m - share
        np.add.at(refs, table[b, :m], 1)
    return dict(refs=refs, table=table, held=held.astype(np.int32))


def _scale_for(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1), and 448 = 0.875 x 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _cache(case, pool, gen, layout):
    """Pages of quantised normals; keys have channels of different strength, as after a projection."""
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    got = []
    both = torch.empty(pool, page, 2, Hkv, D, dtype=torch.float8_e4m3fn, device=DEV) if layout == "fused" else None
    for i, spread in enumerate((0.7, 0.3)):
        strength = torch.exp(spread * torch.randn(Hkv, 1, D, generator=gen, device=DEV))
        if layout == "head":
            codes = torch.empty(pool, Hkv, page, D, dtype=torch.float8_e4m3fn, device=DEV).transpose(1, 2)
        else:
            codes = torch.empty(pool, page, Hkv, D, dtype=torch.float8_e4m3fn, device=DEV) if both is None else both[:, :, i]
        scales = torch.empty(pool, Hkv, dtype=torch.float32, device=DEV)
        step = max(1, (1 << 26) // (Hkv * page * D))
        for lo in range(0, pool, step):
            x = torch.randn(min(step, pool - lo), Hkv, page, D, generator=gen, device=DEV) * strength
            s = _scale_for(x.abs().amax(dim=(2, 3)))
            codes[lo:lo + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).transpose(1, 2)
            scales[lo:lo + step] = s
        got += [codes, scales]
    return got


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 29)
    op = case["op"]
    if own:
        import tree_speculative_verification_attention_gb300 as tsv
    if op == "attention":
        n, start = _lengths(case)
        page, B = case["page"], case["B"]
        offsets = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        pages = -(-(start + n) // page)
        pool = int(pages.sum()) + 2
        ids = np.random.default_rng([int(seed), 13]).permutation(pool).astype(np.int32)
        table = np.full((B, int(pages.max())), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            table[b, :pages[b]] = ids[at:at + pages[b]]
            at += int(pages[b])
        k, ks, v, vs = _cache(case, pool, gen, "head" if case["head_major"] else "token")
        N = int(offsets[-1])
        # rows of a fused projection's output: the queries in front of keys and values
        q = 1.5 * torch.randn(N, case["Hq"] + 2 * case["Hkv"], case["D"], generator=gen, device=DEV)
        q = q.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)[:, :case["Hq"]]
        s = dict(case=case, q=q, k=k, v=v, k_scale=ks, v_scale=vs, table=_put(table), start=_put(start.astype(np.int32)),
                 offsets=_put(offsets), most=int(n.max()), spans=list(zip(offsets.tolist(), n.tolist(), start.tolist())))
        if own:  # what a program keeps: the cache's handle, result buffers, the workspace
            s["cache"] = tsv.PagedCache(k, v, ks, vs)
            s["status"] = torch.zeros(B, dtype=torch.int32, device=DEV)
            s["out"] = torch.empty(q.shape, dtype=q.dtype, device=DEV)
            s["workspace"] = tsv.paged_chunk_attention_workspace(q, s["cache"], B, s["most"])
        return s
    if op == "copy":
        k, ks, v, vs = _cache(case, case["pool"], gen, case["layout"])
        ids = np.random.default_rng([int(seed), 17]).permutation(case["pool"]).astype(np.int32)
        s = dict(case=case, k=k, v=v, k_scale=ks, v_scale=vs, src=_put(np.sort(ids[:case["n"]])), dst=_put(np.sort(ids[case["n"]:2 * case["n"]])))
        if own:
            s["cache"] = tsv.PagedCache(k, v, ks, vs)
            s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    s = {name: _put(a) for name, a in _lists(case, seed).items()}
    s["case"] = case
    if own:
        s["pool"] = tsv.PagePool(s["refs"])
        B, ints = case["B"], lambda size: torch.zeros(size, dtype=torch.int32, device=DEV)  # noqa: E731
        if op == "resize":
            s["status"], s["status_back"] = ints(B), ints(B)
        elif op == "fork":
            s["out"] = dict(copy_src=ints(B), copy_dst=ints(B), status=ints(B))
        else:
            s["out"] = dict(refs=ints(case["pool"]), tables=[torch.full_like(s["table"], -1)], new_id=ints(case["pool"]),
                            move_src=torch.full_like(s["refs"], -1), move_dst=torch.full_like(s["refs"], -1), moved=ints(1), status=ints(1))
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    return {"attention": _attention, "resize": _resize, "fork": _fork, "compact": _compact, "copy": _copy}[state["case"]["op"]](state)


def _rows(codes, scales, ids, rows):
    """The first `rows` rows of the listed pages in fp32, [Hkv, rows, D]."""
    x = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * scales[ids][:, None, :, None]
    return x.flatten(0, 1)[:rows].transpose(0, 1)


def _attention(s):
    case = s["case"]
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        return tsv.paged_chunk_attention(s["q"], s["cache"], s["table"], s["start"], s["offsets"], window=case["window"],
                                         max_rows=s["most"], out=s["out"], workspace=s["workspace"], status=s["status"])[0]
    Hkv, D, G, page, window = case["Hkv"], case["D"], case["Hq"] // case["Hkv"], case["page"], case["window"]
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    for b, (off, n, start) in enumerate(s["spans"]):
        if not n:
            continue
        L = start + n
        ids = s["table"][b, :-(-L // page)].long()
        k, v = _rows(s["k"], s["k_scale"], ids, L), _rows(s["v"], s["v_scale"], ids, L)
        step = max(1, (1 << 28) // (L * Hkv * G))  # rows whose scores are held at once
        for lo in range(0, n, step):
            m = min(step, n - lo)
            q = s["q"][off + lo:off + lo + m].float().view(m, Hkv, G, D).transpose(0, 1).reshape(Hkv, m * G, D)
            scores = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))
            pos = (start + lo + torch.arange(m, device=DEV)).repeat_interleave(G)[:, None]
            key = torch.arange(L, device=DEV)[None, :]
            hide = key > pos
            if window:
                hide = hide | (key <= pos - window)
            scores.masked_fill_(hide[None], -math.inf)
            scores.sub_(scores.amax(dim=-1, keepdim=True)).exp_()
            total = scores.sum(dim=-1, keepdim=True)
            o = (scores @ v) / total
            out[off + lo:off + lo + m] = o.view(Hkv, m, G, D).transpose(0, 1).reshape(m, Hkv * G, D).to(out.dtype)
    return out


def _served(need, refs):
    """Requests in order, as long as the free pages last: which get theirs, and the page ids that they take."""
    free = (refs == 0).nonzero()[:, 0]
    upto = need.cumsum(0)
    got = (upto <= free.shape[0]) | (need == 0)
    return got, free, upto - need


def _give_back(refs, table, first, end):
    """Entries first[b] .. end[b] - 1 of every list: one reference less."""
    i = torch.arange(table.shape[1], device=DEV)[None, :]
    back = table[(i >= first[:, None]) & (i < end[:, None])]
    refs.index_add_(0, back.long(), torch.full_like(back, -1))


def _resize_lists(s, rows):
    """In place; returns the status of each request."""
    refs, table, held, page = s["refs"], s["table"], s["held"], s["case"]["page"]
    want = (rows + (page - 1)) // page
    _give_back(refs, table, want, held)
    need = (want - held).clamp(min=0)
    got, free, before = _served(need, refs)
    i = torch.arange(table.shape[1], device=DEV)[None, :]
    new = got[:, None] & (i >= held[:, None]) & (i < want[:, None])
    take = free[(before[:, None] + i - held[:, None])[new]]
    table[new] = take.to(torch.int32)
    refs[take] = 1
    held.copy_(torch.where(got, want, held))
    return torch.where(got, OK, NO_PAGES).to(torch.int32)


def _resize(s):
    # A step's pages are taken and given back: the pool is as before, the table still shows what was taken.
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        page = s["case"]["page"]
        up = tsv.pages_resize(s["pool"], s["table"], s["held"], s["rows_up"], page, status=s["status"])
        back = tsv.pages_resize(s["pool"], s["table"], s["held"], s["rows"], page, status=s["status_back"])
    else:
        up = _resize_lists(s, s["rows_up"])
        back = _resize_lists(s, s["rows"])
    return {"refs": s["refs"], "table": s["table"], "held": s["held"], "status": up, "status_back": back}


def _fork(s):
    page = s["case"]["page"]
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        r = tsv.pages_fork(s["pool"], s["parents"], s["parent_pages"], s["source"], s["rows"], s["table"], s["held"], page, out=s["out"])
        return {"refs": s["refs"], "table": s["table"], "held": s["held"], **r}
    refs, table, held, rows, source = s["refs"], s["table"], s["held"], s["rows"], s["source"].long()
    _give_back(refs, table, torch.zeros_like(held), held)
    full, part = rows // page, (rows % page > 0).to(torch.int32)
    got, free, before = _served(part, refs)
    i = torch.arange(table.shape[1], device=DEV)[None, :]
    shared = got[:, None] & (i < full[:, None])
    lists = s["parents"][source]
    table[shared] = lists[shared]
    again = lists[shared]
    refs.index_add_(0, again.long(), torch.ones_like(again))
    new = got & (part > 0)
    take = free[before[new]]
    refs[take] = 1
    children = new.nonzero()[:, 0]
    table[children, full[new].long()] = take.to(torch.int32)
    none = torch.full_like(rows, -1)
    src, dst = none.clone(), none.clone()
    src[children] = lists[children, full[new].long()]
    dst[children] = take.to(torch.int32)
    held.copy_(torch.where(got, full + part, torch.zeros_like(held)))
    return {"refs": refs, "table": table, "held": held, "copy_src": src, "copy_dst": dst,
            "status": torch.where(got, OK, NO_PAGES).to(torch.int32)}


def _compact(s):
    refs, table, held = s["refs"], s["table"], s["held"]
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        r = tsv.pages_compact(s["pool"], [table], [held], out=s["out"])
        return {"refs": r["refs"], "table": r["tables"][0], "new_id": r["new_id"], "move_src": r["move_src"], "move_dst": r["move_dst"],
                "moved": r["moved"]}
    pool = refs.shape[0]
    live = refs > 0
    count = live.sum()
    ids = torch.arange(pool, device=DEV)
    src, dst = (live & (ids >= count)).nonzero()[:, 0], (~live & (ids < count)).nonzero()[:, 0]
    new_id = torch.where(live, ids, torch.full_like(ids, -1))
    new_id[src] = dst
    out = refs.clone()
    out[dst] = refs[src]
    out[src] = 0
    fresh = torch.full_like(table, -1)
    inside = torch.arange(table.shape[1], device=DEV)[None, :] < held[:, None]
    fresh[inside] = new_id[table[inside].long()].to(torch.int32)
    moves = []
    for x in (src, dst):  # as long as the pool, -1 behind the moves
        m = torch.full_like(refs, -1)
        m[:x.shape[0]] = x.to(torch.int32)
        moves.append(m)
    return {"refs": out, "table": fresh, "new_id": new_id.to(torch.int32), "move_src": moves[0], "move_dst": moves[1],
            "moved": torch.full((1,), src.shape[0], dtype=torch.int32, device=DEV)}


def _copy(s):
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        tsv.pages_copy(s["cache"], s["src"], s["dst"], status=s["status"])
    else:
        src, dst = s["src"].long(), s["dst"].long()
        for codes, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            codes.view(torch.uint8)[dst] = codes.view(torch.uint8)[src]
            scales[dst] = scales[src]
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------ from the definition


def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(case, prepare(case, seed))
    if case["op"] == "copy":
        s = prepare(case, seed)
        out = {name: s[name].clone() for name in ("k", "v", "k_scale", "v_scale")}
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            for name in out:
                if name in ("k", "v"):
                    out[name].view(torch.uint8)[b].copy_(s[name].view(torch.uint8)[a])
                else:
                    out[name][b].copy_(s[name][a])
        return out
    lists = _lists(case, seed)
    r = {"resize": _exact_resize, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](case, lists)
    return {name: _put(np.asarray(a, dtype=np.int32)) for name, a in r.items()}


def _exact_attention(case, s):
    G, D, page, window = case["Hq"] // case["Hkv"], case["D"], case["page"], case["window"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (off, n, start) in enumerate(s["spans"]):
        for g in range(case["Hkv"]):
            ids = s["table"][b, :-(-(start + n) // page)].long()
            k, v = ((codes[:, :, g].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                     * scales[ids, g].double()[:, None, None]).reshape(-1, D) for codes, scales in
                    ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
            for lo in range(0, n, 512):  # 512 tokens at a time, over the keys that one of them sees
                hi = min(n, lo + 512)
                first, end = max(0, start + lo - window + 1) if window else 0, start + hi
                w = torch.einsum("ngd,ld->ngl", s["q"][off + lo:off + hi, g * G:(g + 1) * G].double(), k[first:end]) / math.sqrt(D)
                at = torch.arange(start + lo, start + hi, device=DEV)[:, None] - torch.arange(first, end, device=DEV)[None, :]
                sees = (at >= 0) & (at < (window or (1 << 40)))
                w = torch.softmax(w.masked_fill(~sees[:, None], -math.inf), dim=-1)
                out[off + lo:off + hi, g * G:(g + 1) * G] = torch.einsum("ngl,ld->ngd", w, v[first:end])
    return out


def _exact_resize(case, lists):
    refs, table, held = (lists[x].tolist() for x in ("refs", "table", "held"))
    status = []
    for rows in (lists["rows_up"].tolist(), lists["rows"].tolist()):
        want = [math.ceil(r / case["page"]) for r in rows]
        for b, w in enumerate(want):
            for i in range(w, held[b]):
                refs[table[b][i]] -= 1
        free = iter([p for p, r in enumerate(refs) if r == 0])
        left = refs.count(0)
        st = []
        for b, w in enumerate(want):
            need = max(0, w - held[b])
            if need and need > left:
                left = -1  # nobody behind takes any
                st.append(NO_PAGES)
                continue
            left -= need
            for i in range(held[b], w):
                table[b][i] = next(free)
                refs[table[b][i]] = 1
            held[b] = w
            st.append(OK)
        status.append(st)
    return {"refs": refs, "table": table, "held": held, "status": status[0], "status_back": status[1]}


def _exact_fork(case, lists):
    refs, table, held, parents = (lists[x].tolist() for x in ("refs", "table", "held", "parents"))
    B = case["B"]
    src, dst, status = [-1] * B, [-1] * B, [OK] * B
    for b in range(B):
        for p in table[b][:held[b]]:
            refs[p] -= 1
    free = [p for p, r in enumerate(refs) if r == 0][::-1]
    over = False
    for b, (f, rows) in enumerate(zip(lists["source"].tolist(), lists["rows"].tolist())):
        full, rest = divmod(rows, case["page"])
        over = over or (rest and not free)
        if over and rest:
            status[b], held[b] = NO_PAGES, 0
            continue
        for i in range(full):
            table[b][i] = parents[f][i]
            refs[parents[f][i]] += 1
        if rest:
            p = free.pop()
            refs[p], table[b][full], src[b], dst[b] = 1, p, parents[f][full], p
        held[b] = full + (1 if rest else 0)
    return {"refs": refs, "table": table, "held": held, "copy_src": src, "copy_dst": dst, "status": status}


def _exact_compact(case, lists):
    refs, pool = lists["refs"].tolist(), case["pool"]
    count = sum(r > 0 for r in refs)
    new_id, out, src, dst = [-1] * pool, [0] * pool, [], []
    hole = 0
    for p, r in enumerate(refs):
        if not r:
            continue
        if p < count:
            new_id[p] = p
        else:
            while refs[hole]:
                hole += 1
            new_id[p] = hole
            src.append(p)
            dst.append(hole)
            hole += 1
        out[new_id[p]] = r
    table = np.full_like(lists["table"], -1)
    back = np.asarray(new_id, dtype=np.int32)
    for b, m in enumerate(lists["held"].tolist()):
        table[b, :m] = back[lists["table"][b, :m]]
    rest = [-1] * (pool - len(src))
    return {"refs": out, "table": table, "new_id": new_id, "move_src": src + rest, "move_dst": dst + rest, "moved": [len(src)]}
