"""Chunk attention on the GPU where one CTA works for longer than any wait may stand still."""
import numpy as np
import pytest
import torch

from test_gpu_paged import dev, i32, make_cache

pytestmark = pytest.mark.gpu


def test_a_tile_that_sits_out_for_longer_than_a_second(tsv):
    """Requests of four tokens behind two million shared keys, then one of 256 tokens: the warps of a unit's second tile have nothing
    to do for more than a second and then go on.  No timeout is reported.  All values are 1, so every output is, off by a weight's
    half step (2^-11) and its own (2^-8)."""
    rng = np.random.default_rng(1)
    page, H, D, B, width = 128, 64, 64, 128, 16384
    cache = make_cache(tsv, rng, 8, page, H, D, True)
    cache.v.view(torch.uint8).fill_(0x38)
    cache.v_scale.fill_(1.0)
    n = np.array([4] * (B - 1) + [256])
    start = np.array([width * page - 64] * (B - 1) + [0])
    offs = np.concatenate([[0], np.cumsum(n)])
    q = torch.randn(int(offs[-1]), H, D, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(torch.bfloat16)
    table = dev(rng.integers(0, 8, size=(B, width)).astype(np.int32))
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    ws = tsv.paged_chunk_attention_workspace(q, cache, B, 256)
    a.record()
    out, st = tsv.paged_chunk_attention(q, cache, table, i32(start), i32(offs), max_rows=256, workspace=ws)
    b.record()
    torch.cuda.synchronize()
    assert (st == 0).all()
    assert ((out.double() - 1).abs() <= 2.0 ** -11 + 2.0 ** -8 + width * page * (2.0 ** -27 + 2.0 ** -28)).all()
    assert a.elapsed_time(b) > 1100.0
