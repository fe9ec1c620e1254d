"""Cases of the paged 8-bit KV cache's operators, and their plain forms.

Four operators: `rope` (rotary positions), `append` (rotate, quantise and write rows into a paged e4m3 cache),
`attention` (token-tree attention over such a cache) and `commit` (the accepted path's rows moved behind the prefix).

The cache: pages of `page` rows, one fp32 power-of-two scale per page and KV head for K and for V; a value is code x scale.
A request's verified rows are the first prefix_len rows of the pages that its row of `table` lists; its speculated tree's
rows are the first rows of the pages that its row of `tree_table` lists.

`run` computes an operator in elementary torch operations in 32 bits (angles in 64), or, with `own` set, calls the framework.
`exact` gives the same outputs from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases


def listed():
    return [
        # Queries of one 20-node tree, 32 heads: one layer's rotation in a verification step (latency counts).
        dict(name="rope-tree20-h32", op="rope", N=20, H=32, D=128, rot=128, interleaved=False, scaling="none", inverse=False,
             dtype="bf16", far=1100, strided=True),
        # Queries of a long prompt chunk, 64 heads, interleaved pairs on half of the head, positions far beyond the trained context.
        dict(name="rope-chunk16384-h64-part", op="rope", N=16384, H=64, D=128, rot=64, interleaved=True, scaling="yarn",
             inverse=False, dtype="bf16", far=131072, strided=False),
        # The gradient of a rotation in fp32, odd sizes, a narrow rotated part.
        dict(name="rope-gradient-f32", op="rope", N=4099, H=9, D=80, rot=20, interleaved=False, scaling="linear", inverse=True,
             dtype="f32", far=9000, strided=False),
        # Keys and values of one 20-node tree, 32 KV heads, into its tree pages.
        dict(name="append-tree20-h32", op="append", B=1, n_lo=20, n_hi=20, p_lo=0, p_hi=0, Hkv=32, D=128, page=16, rot=128,
             interleaved=False, dtype="bf16", head_major=True),
        # Prompt chunks of eight requests of different lengths behind what they hold already, 8 KV heads, 64-row pages.
        dict(name="append-prompts-ragged", op="append", B=8, n_lo=1, n_hi=4096, p_lo=0, p_hi=1000, Hkv=8, D=128, page=64, rot=128,
             interleaved=False, dtype="bf16", head_major=True),
        # One token for each of 8 requests, 64 query / 8 KV heads: plain decoding, no tree.
        dict(name="attn-decode8-gqa64x8", op="attention", B=8, n_lo=1, n_hi=1, p_lo=1000, p_hi=9000, Hq=64, Hkv=8, D=128, page=64,
             tree=False, dtype="bf16", head_major=True),
        # One 20-node tree over a prefix of 1024, 32 heads: one layer of a 7B model's verification step.
        dict(name="attn-llama7b-P1024-n20", op="attention", B=1, n_lo=20, n_hi=20, p_lo=1024, p_hi=1024, Hq=32, Hkv=32, D=128,
             page=16, tree=True, dtype="bf16", head_major=True),
        # 32 requests with 16-node trees over 2048 keys: the cache's bytes are what counts.
        dict(name="attn-batch32-P2048-n16", op="attention", B=32, n_lo=16, n_hi=16, p_lo=2048, p_hi=2048, Hq=32, Hkv=32, D=128,
             page=32, tree=True, dtype="bf16", head_major=True),
        # One 128-node tree over 32768 keys, 64 query / 8 KV heads: 1024 query rows a KV head, the products are what counts.
        dict(name="attn-gqa64x8-P32768-n128", op="attention", B=1, n_lo=128, n_hi=128, p_lo=32768, p_hi=32768, Hq=64, Hkv=8,
             D=128, page=128, tree=True, dtype="bf16", head_major=True),
        # Ragged requests in fp32, heads of 64, token-major pages.
        dict(name="attn-ragged-f32-d64", op="attention", B=3, n_lo=1, n_hi=40, p_lo=0, p_hi=1500, Hq=8, Hkv=2, D=64, page=16,
             tree=True, dtype="f32", head_major=False),
        # The accepted path of one 20-node tree, 32 KV heads.
        dict(name="commit-tree20-h32", op="commit", B=1, n_lo=20, n_hi=20, p_lo=1024, p_hi=1024, Hkv=32, D=128, page=16,
             head_major=True),
        # The accepted paths of 128 requests with trees of up to 256 nodes.
        dict(name="commit-batch128-n256", op="commit", B=128, n_lo=1, n_hi=256, p_lo=0, p_hi=700, Hkv=8, D=128, page=32,
             head_major=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "commit"])
    if op == "rope":
        D = 2 * rng.randint(8, 128)
        H = _log_int(rng, 1, 64)
        N = _log_int(rng, 1, max(1, min(16384, 16384 * 64 * 128 // (H * D * 2))))
        return dict(op=op, N=N, H=H, D=D, rot=2 * rng.randint(1, D // 2), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), inverse=rng.random() < 0.3,
                    dtype=rng.choice(["bf16", "f32"]), far=_log_int(rng, 16, 1 << 20), strided=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 3, 5, 8, 32])
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    common = dict(op=op, Hkv=Hkv, D=D, page=page, head_major=rng.random() < 0.7)
    if op == "append":
        B = _log_int(rng, 1, 32)
        n_hi = _log_int(rng, 1, max(1, 16384 * 8 // (B * Hkv)))
        return dict(common, B=B, n_lo=rng.randint(0, 1), n_hi=n_hi, p_lo=0, p_hi=_log_int(rng, 1, 1000),
                    rot=rng.choice([0, D // 2, D]), interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]))
    if op == "commit":
        return dict(common, B=_log_int(rng, 1, 64), n_lo=1, n_hi=_log_int(rng, 1, 256), p_lo=0, p_hi=_log_int(rng, 1, 700))
    f32 = rng.random() < 0.15
    tree = rng.random() < 0.7
    G = rng.choice([1, 2, 3, 4, 7, 8])
    B = _log_int(rng, 1, 4 if f32 else 32)
    n_hi = _log_int(rng, 1, 40 if f32 else max(1, min(256, 1024 // (G * min(B, 8))))) if tree else 1
    most = min(32768, 32 * 2048 * 32 // (B * max(Hkv, 4)), 32768 * 8 * 1024 // (Hkv * n_hi * G * B))
    p_hi = _log_int(rng, 1, 1500) if f32 else _log_int(rng, 16, max(16, most))
    return dict(common, B=B, n_lo=1, n_hi=n_hi, p_lo=rng.choice([0, p_hi // 4, p_hi]), p_hi=p_hi, Hq=G * Hkv, tree=tree,
                dtype="f32" if f32 else "bf16")


# ------------------------------------------------------------------ what a pass cannot do without


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    op = case["op"]
    if op == "rope":
        vals = case["N"] * case["H"] * case["D"]
        return {"bytes": 2 * vals * _size(case["dtype"]) + 4 * case["N"], "flops": 3 * case["N"] * case["H"] * case["rot"]}
    lay = _layout(case, 0)
    HD, Hkv = case["Hkv"] * case["D"], case["Hkv"]
    N, pages = int(lay["offsets"][-1]), 0
    if op == "append":
        for p, n in zip(lay["prefix"].tolist(), lay["nodes"].tolist()):
            if n:
                pages += (p + n - 1) // case["page"] - p // case["page"] + 1
        return {"bytes": 2 * N * HD * (_size(case["dtype"]) + 1) + 8 * pages * Hkv, "flops": 2 * 4 * N * HD}
    if op == "commit":
        rows = sum(int(a) + 1 for a in lay["accept"])
        return {"bytes": 2 * 2 * rows * HD, "flops": 2 * 2 * rows * HD}
    keys = sum(int(p) + (int(n) if case["tree"] else 0) for p, n in zip(lay["prefix"], lay["nodes"]))
    seen = sum(int(n) * int(p) for p, n in zip(lay["prefix"], lay["nodes"]))
    if case["tree"]:
        seen += int(lay["ancestors"].sum())
    return {"bytes": 2 * keys * HD + 2 * N * case["Hq"] * case["D"] * _size(case["dtype"]),
            "flops": 4 * seen * case["Hq"] * case["D"]}


# ------------------------------------------------------------------ inputs


def _layout(case, seed):
    """Host side of a batch: lengths, trees, accepted paths, page tables (all from the seed)."""
    rng = np.random.default_rng([int(seed), 7])
    B, page = case["B"], case["page"]
    lay_rng = np.random.default_rng([1, B, case["n_hi"], case["p_hi"]])  # lengths belong to the case
    nodes = lay_rng.integers(case["n_lo"], case["n_hi"] + 1, size=B)
    nodes[0] = max(nodes[0], 1)
    prefix = lay_rng.integers(case["p_lo"], case["p_hi"] + 1, size=B)
    offsets = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    N = int(offsets[-1])
    parent = np.full(N, -1, dtype=np.int32)
    depth = np.zeros(N, dtype=np.int32)
    path = np.full(N, -1, dtype=np.int32)
    accept = np.zeros(B, dtype=np.int32)
    most = int(max(nodes)) if B else 0
    anc = np.zeros((N, min(most, 256)), dtype=bool)
    tree = case["op"] == "commit" or case.get("tree", False)
    for b in range(B):
        o, n = int(offsets[b]), int(nodes[b])
        if not n or not tree:
            continue
        for i in range(1, n):
            low = max(0, i - 1 - i // 3)
            parent[o + i] = lay_rng.integers(low, i)  # the newest third: deep paths and many branches
            depth[o + i] = depth[o + parent[o + i]] + 1
        for i in range(n):
            if i:
                anc[o + i] = anc[o + parent[o + i]]
            anc[o + i, i] = True
        leaf = int(lay_rng.integers(0, n))
        way = [leaf]
        while way[-1]:
            way.append(int(parent[o + way[-1]]))
        path[o:o + len(way)] = way[::-1]
        accept[b] = len(way) - 1
    grown = prefix + (nodes if case["op"] == "append" else accept + 1 if case["op"] == "commit" else 0)
    main_pages, tree_pages = -(-grown // page), -(-nodes // page) if tree else np.zeros(B, dtype=np.int64)
    pool = int(main_pages.sum() + tree_pages.sum()) + 2
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((B, max(1, int(main_pages.max()))), -1, dtype=np.int32)
    tree_table = np.full((B, max(1, int(tree_pages.max()))), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :main_pages[b]] = ids[at:at + main_pages[b]]
        at += int(main_pages[b])
        tree_table[b, :tree_pages[b]] = ids[at:at + tree_pages[b]]
        at += int(tree_pages[b])
    words = np.zeros((N, 8), dtype=np.uint32)
    for j in range(anc.shape[1]):
        words[:, j >> 5] |= anc[:, j].astype(np.uint32) << np.uint32(j & 31)
    return dict(prefix=prefix.astype(np.int32), nodes=nodes, offsets=offsets, parent=parent, depth=depth, path=path, accept=accept,
                ancestors=anc, words=words.view(np.int32), table=table, tree_table=tree_table, pool=pool)


def _frequencies(rot, scaling):
    """inverse frequencies in 64 bits and the amplitude: base 10000, trained on 4096 positions, four times that wanted."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    base, factor, trained = 10000.0, 4.0, 4096.0
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / max(rot, 1))
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        low = rot * math.log(trained / (32.0 * 2 * math.pi)) / (2 * math.log(base))
        high = rot * math.log(trained / (1.0 * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rot - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        return f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _put(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _cache(case, pool, gen):
    """A pool of pages of quantised normals; keys have channels of different strength, as after a projection."""
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    got = []
    for spread in (0.7, 0.3):
        strength = torch.exp(spread * torch.randn(Hkv, 1, D, generator=gen, device=DEV))
        codes = torch.empty(pool, Hkv, page, D, dtype=torch.float8_e4m3fn, device=DEV)
        scales = torch.empty(pool, Hkv, dtype=torch.float32, device=DEV)
        step = max(1, (1 << 26) // (Hkv * page * D))
        for lo in range(0, pool, step):
            x = torch.randn(min(step, pool - lo), Hkv, page, D, generator=gen, device=DEV) * strength
            s = _scale_for(x.abs().amax(dim=(2, 3)))
            codes[lo:lo + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
            scales[lo:lo + step] = s
        codes = codes.transpose(1, 2)  # [page id, row, head, d]
        got += [codes if case["head_major"] else codes.contiguous(), scales]
    return got


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 17)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    if case["op"] == "rope":
        f, amplitude = _frequencies(case["rot"], case["scaling"])
        x = normal(case["N"], case["H"] + (2 if case["strided"] else 0), case["D"]).to(_type(case))
        pos = torch.randint(0, case["far"], (case["N"],), generator=gen, device=DEV, dtype=torch.int32)
        s = dict(case=case, x=x[:, :case["H"]], positions=pos, inv_freq=f.to(DEV), amplitude=amplitude)
        if own:  # the buffer that a program's layers share
            s["out"] = torch.empty(s["x"].shape, dtype=s["x"].dtype, device=DEV)
        return s
    lay = _layout(case, seed)
    N, Hkv, D = int(lay["offsets"][-1]), case["Hkv"], case["D"]
    k, ks, v, vs = _cache(case, lay["pool"], gen)
    s = dict(case=case, k=k, v=v, k_scale=ks, v_scale=vs, table=_put(lay["table"]), tree_table=_put(lay["tree_table"]),
             prefix=_put(lay["prefix"]), offsets=_put(lay["offsets"]), most_nodes=int(max(lay["nodes"])),
             request=_put(np.repeat(np.arange(case["B"]), lay["nodes"])), local=_put(np.arange(N) - np.repeat(lay["offsets"][:-1], lay["nodes"])))
    if case["op"] == "append":
        # rows of a fused projection's output: K and V side by side
        kv = normal(N, 2, Hkv, D).to(_type(case))
        f, amplitude = _frequencies(case["rot"], "none")
        s.update(k_new=kv[:, 0], v_new=kv[:, 1], inv_freq=f.to(DEV) if case["rot"] else None, amplitude=amplitude,
                 positions=(s["prefix"][s["request"]] + s["local"]).to(torch.int32))
    elif case["op"] == "commit":
        s.update(path=_put(lay["path"]), accept=_put(lay["accept"]))
    else:
        s.update(q=(1.5 * normal(N, case["Hq"], D)).to(_type(case)), anc=_put(lay["words"]), most_prefix=int(max(lay["prefix"])))
    if own:  # what a program keeps: the cache's handle, result buffers, the workspace
        import tree_speculative_verification_attention_gb300 as tsv

        s["cache"] = tsv.PagedCache(k, v, ks, vs)
        s["status"] = torch.zeros(case["B"], dtype=torch.int32, device=DEV)
        if case["op"] == "attention":
            s["out"] = torch.empty_like(s["q"])
            s["workspace"] = tsv.paged_tree_attention_workspace(s["q"], s["cache"], case["B"], s["most_nodes"])
        if case["op"] == "commit":
            s["result"] = dict(new_len=torch.empty(case["B"], dtype=torch.int32, device=DEV), status=s["status"])
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    return {"rope": _rope, "append": _append, "attention": _attention, "commit": _commit}[state["case"]["op"]](state)


def _scale_for(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1), and 448 = 0.875 x 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _rows(codes, *index):
    """codes[index] in fp32."""
    return codes.view(torch.uint8)[index].view(torch.float8_e4m3fn).float()


def _set_rows(codes, values, *index):
    codes.view(torch.uint8)[index] = values.to(torch.float8_e4m3fn).view(torch.uint8)


def _rotate(x, positions, inv_freq, amplitude, interleaved, inverse):
    x = x.float()
    if inv_freq is None:
        return x
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq
    c, s = (amplitude * angle.cos()).float()[:, None], (amplitude * angle.sin()).float()[:, None]
    if inverse:
        s = -s
    part = x[..., :2 * half]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    a, b = a * c - b * s, b * c + a * s
    both = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((both, x[..., 2 * half:]), dim=-1)


def _rope(s):
    case = s["case"]
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        return tsv.rope(s["x"], s["positions"], s["inv_freq"], interleaved=case["interleaved"], inverse=case["inverse"],
                        amplitude=s["amplitude"], out=s["out"])
    y = _rotate(s["x"], s["positions"], s["inv_freq"], s["amplitude"], case["interleaved"], case["inverse"])
    return y.to(s["x"].dtype)


def _write_rows(codes, scales, x, table, start, request, row, page):
    """Rows `x` [N, Hkv, D] (fp32) into rows start[b] + row of request b's pages, under the pages' scales."""
    if not x.shape[0]:
        return
    B, width = table.shape
    at = start[request].long() + row.long()
    slot = request.long() * width + at // page  # a page of a request, by its place in the table
    Hkv = x.shape[1]
    amax = torch.zeros(B * width, Hkv, device=x.device).scatter_reduce_(
        0, slot[:, None].expand(-1, Hkv), x.abs().amax(dim=-1), "amax", include_self=True)
    touched = torch.zeros(B * width, dtype=torch.bool, device=x.device)
    touched[slot] = True
    slots = touched.nonzero()[:, 0]
    ids = table.reshape(-1)[slots].long()
    first = (slots % width) * page  # the page's first row in its request
    kept = (start.long()[slots // width] - first).clamp(0, page)
    old, need = scales[ids], _scale_for(amax[slots])
    new = torch.where((kept > 0)[:, None], torch.maximum(old, need), need)
    was = _rows(codes, ids)
    again = (was * (old / new)[:, None, :, None]).to(torch.float8_e4m3fn).float()
    keep = torch.arange(page, device=x.device)[None, :] < kept[:, None]
    _set_rows(codes, torch.where(keep[:, :, None, None], again, was), ids)
    scales[ids] = new
    pid = table.reshape(-1)[slot].long()
    _set_rows(codes, x / scales[pid][:, :, None], pid, at % page)


def _append(s):
    case = s["case"]
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        tsv.paged_append(s["cache"], s["table"], s["k_new"], s["v_new"], s["offsets"], start=s["prefix"],
                         positions=s["positions"], inv_freq=s["inv_freq"], interleaved=case["interleaved"],
                         amplitude=s["amplitude"], max_rows=s["most_nodes"], status=s["status"])
    else:
        k = _rotate(s["k_new"], s["positions"], s["inv_freq"], s["amplitude"], case["interleaved"], False)
        _write_rows(s["k"], s["k_scale"], k, s["table"], s["prefix"], s["request"], s["local"], case["page"])
        _write_rows(s["v"], s["v_scale"], s["v_new"].float(), s["table"], s["prefix"], s["request"], s["local"], case["page"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _gather(codes, scales, table, rows):
    """[B, pages x page, Hkv, D] in fp32 of the first `rows` rows of each request's pages."""
    page = codes.shape[1]
    ids = table[:, :-(-rows // page)].long().clamp(min=0)
    x = _rows(codes, ids) * scales[ids][:, :, None, :, None]
    return x.flatten(1, 2)[:, :rows]


def _attention(s):
    case = s["case"]
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        out, _ = tsv.paged_tree_attention(s["q"], s["cache"], s["table"], s["prefix"], s["offsets"],
                                          tree_table=s["tree_table"] if case["tree"] else None,
                                          anc=s["anc"] if case["tree"] else None, max_nodes=s["most_nodes"], out=s["out"],
                                          workspace=s["workspace"], status=s["status"])
        return out
    B, Hkv, D, G, n, P = case["B"], case["Hkv"], case["D"], case["Hq"] // case["Hkv"], s["most_nodes"], max(1, s["most_prefix"])
    request, local = s["request"].long(), s["local"].long()
    k, v = _gather(s["k"], s["k_scale"], s["table"], P), _gather(s["v"], s["v_scale"], s["table"], P)
    seen = (torch.arange(P, device=DEV)[None, :] < s["prefix"][:, None])[:, None, :].expand(B, n, P)
    if case["tree"]:
        k = torch.cat((k, _gather(s["k"], s["k_scale"], s["tree_table"], n)), dim=1)
        v = torch.cat((v, _gather(s["v"], s["v_scale"], s["tree_table"], n)), dim=1)
        j = torch.arange(n, device=DEV)
        bits = torch.zeros(B, n, n, dtype=torch.bool, device=DEV)
        bits[request, local] = ((s["anc"][:, j // 32] >> (j % 32).to(torch.int32)) & 1).bool()
        seen = torch.cat((seen, bits), dim=2)
    q = torch.zeros(B, n, Hkv, G, D, device=DEV)
    q[request, local] = s["q"].float().view(-1, Hkv, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    scores = (q @ k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    hide = ~seen.repeat_interleave(G, dim=1)[:, None]
    scores.masked_fill_(hide, -math.inf)
    top = scores.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    scores.sub_(top).exp_()
    total = scores.sum(dim=-1, keepdim=True)
    o = (scores @ v.permute(0, 2, 1, 3)) / total.clamp(min=1e-30)
    o = o.view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hkv * G, D)
    return o[request, local].to(s["q"].dtype)


def _commit(s):
    case = s["case"]
    if own:
        import tree_speculative_verification_attention_gb300 as tsv

        new_len = tsv.paged_commit(s["cache"], s["table"], s["tree_table"], s["prefix"], s["offsets"], s["path"], s["accept"],
                                   max_nodes=s["most_nodes"], out=s["result"])["new_len"]
    else:
        page = case["page"]
        hit = s["path"] >= 0
        request, row, node = s["request"][hit], s["local"][hit], s["path"][hit].long()
        ids = s["tree_table"][request.long(), node // page].long()
        for codes, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            x = _rows(codes, ids, node % page) * scales[ids][:, :, None]
            _write_rows(codes, scales, x, s["table"], s["prefix"], request, row, page)
        new_len = s["prefix"] + 1 + s["accept"]
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "new_len": new_len}


# ------------------------------------------------------------------ from the definition, in 64 bits


def _power(e):
    """2^e in 64 bits, to the last bit (from its exponent field)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """The nearest multiple of the step at |x| (ties to even): 3 bits behind the leading one, none below 2^-9."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -20))
    step = _power((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _smallest_power(amax):
    some = amax > 0
    e = torch.ceil(torch.log2(torch.where(some, amax, torch.ones_like(amax)) / E4M3_MAX)).to(torch.int64)
    e = torch.where(amax <= E4M3_MAX * _power(e - 1), e - 1, e)  # the logarithm may be off by its last bit
    e = torch.where(amax > E4M3_MAX * _power(e), e + 1, e)
    return _power(torch.where(some, e, torch.full_like(e, -126)).clamp(min=-126))


def _exact_rows(codes, scales, rows_of, table, start, page):
    """Request by request and page by page."""
    for b, x in enumerate(rows_of):
        done, p0 = 0, int(start[b])
        while done < x.shape[0]:
            at = p0 + done
            pid, r = int(table[b, at // page]), at % page
            m = min(page - r, x.shape[0] - done)
            part = x[done:done + m]
            s = _smallest_power(part.abs().amax(dim=(0, 2)))
            if r > 0 and done == 0:
                grown = torch.maximum(s, scales[pid])
                codes[pid, :r] = _round_e4m3(codes[pid, :r] * (scales[pid] / grown)[None, :, None])
                s = grown
            codes[pid, r:r + m] = _round_e4m3(part / s[None, :, None])
            scales[pid] = s
            done += m


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s["x"].double(), s, case)
    offs = s["offsets"].tolist()
    if case["op"] in ("append", "commit"):
        K, V, KS, VS = s["k"].double(), s["v"].double(), s["k_scale"].double(), s["v_scale"].double()
        table, start, page = s["table"].tolist(), s["prefix"].tolist(), case["page"]
        table = np.asarray(table)
        if case["op"] == "append":
            k = s["k_new"].double()
            if case["rot"]:
                k = _exact_rope(k, s, dict(case, inverse=False))
            v = s["v_new"].double()
            ks, vs = [k[a:b] for a, b in zip(offs, offs[1:])], [v[a:b] for a, b in zip(offs, offs[1:])]
            new_len = None
        else:
            path, accept, tt = s["path"].tolist(), s["accept"].tolist(), s["tree_table"].tolist()
            ks, vs = [], []
            for b in range(case["B"]):
                way = path[offs[b]:offs[b] + accept[b] + 1]
                ids = [tt[b][i // page] for i in way]
                rows = [i % page for i in way]
                ks.append(K[ids, rows] * KS[ids][:, :, None])
                vs.append(V[ids, rows] * VS[ids][:, :, None])
            new_len = torch.tensor([p + 1 + a for p, a in zip(start, accept)], dtype=torch.int32)
        _exact_rows(K, KS, ks, table, start, page)
        _exact_rows(V, VS, vs, table, start, page)
        out = {"k": K, "v": V, "k_scale": KS, "v_scale": VS}
        return out if new_len is None else dict(out, new_len=new_len)
    G, D, page = case["Hq"] // case["Hkv"], case["D"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    parent = _layout(case, seed)["parent"]
    prefix, table, tree = s["prefix"].tolist(), s["table"].long(), s["tree_table"].long()
    for b in range(case["B"]):
        n, P = offs[b + 1] - offs[b], prefix[b]
        ids = table[b, :-(-P // page)]
        mask = torch.zeros(n, P + (n if case["tree"] else 0), dtype=torch.bool)
        mask[:, :P] = True
        if case["tree"]:
            for i in range(n):
                j = i
                while j >= 0:
                    mask[i, P + j] = True
                    j = int(parent[offs[b] + j])
        mask = mask.to(DEV)
        for g in range(case["Hkv"]):
            def rows_of(codes, scales):
                x = (_rows(codes, ids)[:, :, g].double() * scales[ids, g].double()[:, None, None]).reshape(-1, D)[:P]
                if case["tree"]:
                    more = tree[b, :-(-n // page)]
                    y = (_rows(codes[:, :, g], more).double() * scales[more, g].double()[:, None, None]).reshape(-1, D)[:n]
                    x = torch.cat((x, y))
                return x
            k, v = rows_of(s["k"], s["k_scale"]), rows_of(s["v"], s["v_scale"])
            if not k.shape[0]:
                continue
            q = s["q"][offs[b]:offs[b + 1], g * G:(g + 1) * G].double()
            w = torch.einsum("ngd,ld->ngl", q, k) / math.sqrt(D)
            w = w.masked_fill(~mask[:, None], -math.inf)
            w = torch.softmax(w, dim=-1) if P or case["tree"] else w * 0
            out[offs[b]:offs[b + 1], g * G:(g + 1) * G] = torch.einsum("ngl,ld->ngd", w, v)
    return out


def _exact_rope(x, s, case):
    """Each pair as a complex number times amplitude x exp(+-i angle)."""
    half = s["inv_freq"].numel()
    angle = s["positions"].double()[:, None, None] * s["inv_freq"]
    if case["inverse"]:
        angle = -angle
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle)
    if case["interleaved"]:
        z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:-1], half, 2).contiguous()) * turn
        part = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
        part = torch.cat((z.real, z.imag), dim=-1)
    return torch.cat((part, x[..., 2 * half:]), dim=-1)
