"""Pins of the paged cache's 64-bit reference (CPU): e4m3 rounding against torch's conversion, scales, rotations."""
import math

import numpy as np
import torch

import _paged_ref as R


def test_e4m3_values_match_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(R.VALUES))
    assert np.array_equal(t[~np.isnan(t)], R.VALUES[~np.isnan(t)])


def test_rounding_matches_torch_and_ties_go_to_even():
    rng = np.random.default_rng(0)
    v = np.sort(R.VALUES[:127])
    mid = (v[1:] + v[:-1]) / 2  # every tie
    x = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), rng.normal(size=4000) * 50]).astype(np.float32)
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    ok = np.abs(x) <= 448
    assert np.array_equal(R.round_e4m3(x)[ok], want[ok])
    assert R.round_e4m3(np.inf) == 448 and R.round_e4m3(-1e9) == -448 and np.isnan(R.round_e4m3(np.nan))


def test_scale_is_the_smallest_power_of_two():
    for a in (1e-30, 0.3, 1.0, 1.75, 1.7500001, 3.5, 448.0, 448.1, 6e4, 3e38):
        s = R.scale_for(a)
        assert math.log2(s) == int(math.log2(s)) and a <= 448 * s and a > 448 * s / 2
    assert R.scale_for(0.0) == 2.0 ** -126 and R.scale_for(1e-44) == 2.0 ** -126


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(1)
    x, pos, w = rng.normal(size=(5, 2, 12)), np.array([0, 1, -3, 77, 1000]), np.array([1.0, 0.3, 0.01])
    for inter in (False, True):
        y = R.rotate(x, pos, w, interleaved=inter, amplitude=1.5)
        a, b = (x[..., :6:2], x[..., 1:6:2]) if inter else (x[..., :3], x[..., 3:6])
        z = (a + 1j * b) * 1.5 * np.exp(1j * pos[:, None, None] * w)
        ya, yb = (y[..., :6:2], y[..., 1:6:2]) if inter else (y[..., :3], y[..., 3:6])
        assert np.allclose(ya, z.real, atol=1e-12) and np.allclose(yb, z.imag, atol=1e-12)
        assert np.array_equal(y[..., 6:], x[..., 6:])
        back = R.rotate(y, pos, w, interleaved=inter, inverse=True, amplitude=1 / 1.5)
        assert np.allclose(back, x, atol=1e-12)


def test_attention_by_hand():
    """Two keys with scores 0 and ln 3 (after the scale): weights 1/4 and 3/4."""
    k = np.zeros((1, 16, 1, 64))
    v = np.zeros((1, 16, 1, 64))
    k[0, 1, 0, 0] = 2.0
    v[0, 0, 0, :] = 4.0
    v[0, 1, 0, :] = -8.0
    c = R.Cache(k, v, np.ones((1, 1)), np.full((1, 1), 0.5))
    q = np.zeros((1, 1, 64))
    q[0, 0, 0] = math.log(3.0)
    out, spread, size = R.attention(q, c, [[0]], [2], [0, 1], scale=0.5)
    assert np.allclose(out, 0.25 * 2.0 - 0.75 * 4.0) and np.allclose(spread, 0.25 * 2 + 0.75 * 4)
    assert np.allclose(size, math.log(3.0))
    out, _, _ = R.attention(q, c, [[0]], [0], [0, 1], scale=0.5)
    assert np.array_equal(out, np.zeros((1, 1, 64)))
