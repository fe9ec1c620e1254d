"""Verification beside the call before it (tsv_set_verify_overlap): what it must still come behind."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("between", ["prepare", "attention", "commit", "expand", "merge"])
def test_verification_comes_behind_the_call_before_the_last(tsv, between):
    """A rotation by 0 writes the logits in one long wave of blocks, a small call follows, then the verification, which may run
    beside the small call but reads what the rotation wrote."""
    B, n, V = 19, 128, 65536
    N = B * n
    want = torch.randn(N, V, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    logits = torch.empty_like(want)
    parent, offs = i32(np.tile(np.arange(-1, n - 1), B)), i32(np.arange(B + 1) * n)
    tokens = torch.cat([want[:1].argmax(-1), want.argmax(-1)[:-1]]).int()  # every node accepted
    zeros, freq = i32(np.zeros(N)), tsv.rope_frequencies(1024, device="cuda")[0]
    h = tsv.handle()
    ws = torch.zeros(tsv.tsv_tree_verify_greedy_workspace_size(h, B, N, V), dtype=torch.uint8, device="cuda")
    g = tsv.tree_verify_greedy(want, tokens, parent, offs, workspace=ws)
    assert (g["accept_len"] == n - 1).all()
    p, o, st = i32([-1, 0, 1]), i32([0, 3]), i32([0])
    anc, depth = torch.empty(3, 8, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    kv = torch.randn(2, 1, 8, 2, 64, device="cuda")
    q, out, plen = torch.randn(3, 2, 64, device="cuda"), torch.empty(3, 2, 64, device="cuda"), i32([4])
    some, picked = torch.randn(3, 50, device="cuda"), torch.empty(3, 2, dtype=torch.int32, device="cuda")
    m = tsv.tree_merge(p, p + 1, o, i32([0, 1]))
    calls = {
        "prepare": lambda: tsv.tsv_tree_prepare(h, p, o, 1, anc, depth, st),
        "attention": lambda: tsv.tree_attention(q, kv[0], kv[1], [4], [0, 3], plen, o, parent=p, out=out, status=st,
                                                workspace=ws_a),
        "commit": lambda: tsv.tsv_kv_commit(h, tsv.TSV_F32, kv[0], kv[1], *kv[0].stride()[:3], 1, 2, 64, plen, o, i32_path, last,
                                            new, st),
        "expand": lambda: tsv.tsv_tree_expand(h, some, 50, 3, 2, picked),
        "merge": lambda: tsv.tsv_tree_merge(h, p, tok3, o, one_tree, 1, m["parent"], m["tokens"], m["source"], m["count"], m["status"]),
    }
    ws_a = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    i32_path, last, new, tok3, one_tree = i32([0, 1, 2]), i32([2]), i32([0]), p + 1, i32([0, 1])
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
