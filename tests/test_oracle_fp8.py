"""Pins of the 8-bit oracle: the E4M3 grid, nearest codes by brute force, the scale rule by its
inequality, and the norm's formula."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8


def test_grid_is_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.isnan(t), np.isnan(fp8.VALUES))
    ok = ~np.isnan(t)
    np.testing.assert_array_equal(t[ok], fp8.VALUES[ok])
    assert fp8.VALUES[0x7E] == 448.0 and fp8.VALUES[1] == 2.0 ** -9


def test_codes_are_nearest_and_ties_even():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 2000), np.ldexp(rng.standard_normal(2000), -6),
                        fp8._MID, -fp8._MID, fp8._MAG, -fp8._MAG])
    got = fp8.codes_of(v)
    dist = np.abs(v[:, None] - np.where(np.isnan(fp8.VALUES), np.inf, fp8.VALUES)[None, :])
    best = dist.min(1)
    np.testing.assert_array_equal(dist[np.arange(v.size), got], best)
    tied = np.isin(np.abs(v), fp8._MID)
    assert np.all(got[tied] % 2 == 0)
    np.testing.assert_array_equal(got >> 7, np.signbit(v).astype(np.uint8))


@pytest.mark.parametrize("amax", [448.0, 448.0 * (1 + 2.0 ** -23), 1.0, 1.75, 1.7500001, 2.0 ** -133, 3.4e38, 1e-30])
def test_exponent_rule(amax):
    e = fp8.exponent_of(amax)
    assert amax <= math.ldexp(448.0, e)
    assert e == -127 or amax > math.ldexp(448.0, e - 1)
    assert 0 <= e + 127 <= 247


def test_blocks_and_short_last_block():
    rng = np.random.default_rng(1)
    X = rng.standard_normal((3, 160)) * np.exp(rng.standard_normal((3, 1)))
    X[1, :128] = 0
    X[2, 140] = np.inf
    c, s = fp8.encode_rows(X)
    assert s.shape == (3, 2) and s[1, 0] == 0 and np.all(c[1, :128] == 0)
    assert s[2, 1] == 0xFF and np.all(c[2, 128:] == 0x7F) and s[2, 0] != 0xFF
    D = fp8.decode_rows(c, s)
    fine = np.isfinite(D)
    step = np.ldexp(1.0, np.repeat(s.astype(int) - 127, 128, 1)[:, :160] - 10)
    assert np.all(np.abs(D - X)[fine] <= (2.0 ** -4 * np.abs(X) + step)[fine])
    W = rng.standard_normal((160, 144))
    wc, ws = fp8.encode_weight(W)
    assert wc.shape == (144, 160) and ws.shape == (2, 2)
    for i in range(2):
        for j in range(2):
            top = np.abs(W.T[128 * i:128 * i + 128, 128 * j:128 * j + 128]).max()
            assert ws[i, j] == fp8.exponent_of(top) + 127


def test_norm_formula():
    rng = np.random.default_rng(2)
    x, r = rng.standard_normal((4, 96)), rng.standard_normal((4, 96))
    g = rng.standard_normal(96)
    y, res = fp8.rmsnorm(x, g, 1e-5, r)
    h = x + r
    ref = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5) * g
    np.testing.assert_allclose(y, ref, rtol=6 * 2.0 ** -24, atol=2e-6)   # x, r, h, root, 2 products in fp32
    np.testing.assert_allclose(res, h, rtol=2.0 ** -22, atol=1e-6)
    y0, none = fp8.rmsnorm(np.zeros((2, 96)), g, 1e-5)
    assert none is None and np.all(y0 == 0)


def test_activations():
    z = np.array([-800.0, -5.0, 0.0, 1.0, 30.0])
    t = torch.from_numpy(z)
    np.testing.assert_allclose(fp8.activation(z), torch.nn.functional.silu(t).numpy(), rtol=1e-14, atol=1e-300)
    np.testing.assert_allclose(fp8.activation(z, "gelu"), torch.nn.functional.gelu(t).numpy(), rtol=1e-9, atol=1e-12)
