"""The 64-bit oracle of the embedding and of MXFP4 against the definitions:
the nearest value of the grid by search over all of it, the properties of the
block scales, and matrix products."""
import math

import numpy as np
import pytest

from oracle import layers

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def test_values_of_all_codes():
    codes = np.arange(16, dtype=np.uint8)[None]
    for s in (1, 127, 200, 254):
        got = layers.mxfp4_values(codes, np.array([[s]], dtype=np.uint8))[0]
        assert got.tolist() == [math.ldexp(v, s - 127) for v in GRID + [-g for g in GRID]]
    assert np.isnan(layers.mxfp4_values(codes, np.array([[255]], dtype=np.uint8))).all()


def test_nearest_of_the_grid_ties_to_even():
    """With 4 in the block its scale is one, and values are those of the grid."""
    for k in range(-7 * 64, 7 * 64 + 1):
        t = k / 64
        codes, scales = layers.mxfp4_quantize(np.array([[4.0, t]]))
        assert scales[0, 0] == 127
        got = float(layers.mxfp4_values(codes, scales)[0, 1])
        best = min(abs(abs(t) - g) for g in GRID)
        near = [i for i, g in enumerate(GRID) if abs(abs(t) - g) == best]
        want = GRID[min(near, key=lambda i: i % 2)]       # of two neighbours, the even code
        assert abs(got) == want and (got == 0 or (got < 0) == (t < 0)), t


@pytest.mark.parametrize("noise", [False, True])
def test_scales_put_the_largest_into_the_grid(noise):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(50, 100)) * 10.0 ** rng.uniform(-30, 30, size=(50, 1))
    r = rng.integers(0, 256, size=x.shape) if noise else None
    codes, scales = layers.mxfp4_quantize(x, r)
    for i in range(50):
        for b in range(4):
            t = np.max(np.abs(x[i, 32 * b:32 * b + 32])) * 2.0 ** (127 - float(scales[i, b]))
            assert (3 < t <= 6) if noise else (4 <= t < 8)
    v = layers.mxfp4_values(codes, scales)
    step = np.where(np.abs(v) < 2, 1, 1) * 2.0 ** (np.repeat(scales, 32, 1)[:, :100].astype(float) - 127)
    assert np.all(np.abs(v - x) <= (2 if noise else 2) * step)


def test_noise_rounds_up_in_proportion():
    """Over all 256 bytes a value is rounded up in proportion, to 1 / 512."""
    r = np.arange(256)[:, None].repeat(2, 1)
    for t in (0.1, 0.3, 0.5, 0.77, 1.26, 2.4, 3.9, 4.5, 5.99, 6.0):
        x = np.tile([6.0, -t], (256, 1))
        codes, scales = layers.mxfp4_quantize(x, r)
        assert (scales == 127).all()
        v = layers.mxfp4_values(codes, scales)
        assert (v[:, 0] == 6).all()
        gap = 0.5 if t < 2 else 1.0 if t < 4 else 2.0
        assert abs(v[:, 1].mean() + t) <= gap / 512 + 1e-12


def test_blocks_that_stand_for_nothing_finite():
    for bad in (math.inf, -math.inf, math.nan):
        x = np.ones((2, 70))
        x[1, 40] = bad
        codes, scales = layers.mxfp4_quantize(x)
        v = layers.mxfp4_values(codes, scales)
        assert scales.tolist() == [[125, 125, 125], [125, 255, 125]] and (codes[1, 32:64] == 0).all()
        assert np.isnan(v[1, 32:64]).all() and np.isfinite(np.delete(v[1], range(32, 64))).all()
    codes, scales = layers.mxfp4_quantize(np.zeros((1, 5)))
    assert (codes == 0).all() and scales.tolist() == [[0]]


def test_embedding_is_a_product_with_indicators():
    rng = np.random.default_rng(6)
    tokens = np.array([[3, -1, 0, 3], [7, 2, 100, 3]])
    w, g = rng.normal(size=(8, 5)), rng.normal(size=(2, 4, 5))
    one = np.zeros((8, 8))
    for i, t in enumerate(tokens.reshape(-1)):
        if 0 <= t < 8:
            one[i, t] = 1
    assert np.allclose(layers.embedding(tokens, w, 3.0).reshape(8, 5), 3 * one @ w, rtol=1e-14)
    sums, sizes, n = layers.embedding_grad(tokens, g, 8, 3.0)
    assert np.allclose(sums, 3 * one.T @ g.reshape(8, 5), rtol=1e-14)
    assert np.allclose(sizes, 3 * one.T @ np.abs(g.reshape(8, 5)), rtol=1e-14)
    assert n.tolist() == one.sum(0).astype(int).tolist()


def test_embedding_gradient_by_differences():
    """The gradient of sum(out * g) is the difference quotient (the function is
    linear, so it is exact up to rounding)."""
    rng = np.random.default_rng(7)
    tokens, w, g = np.array([1, 4, 1, -1, 2, 9]), rng.normal(size=(5, 3)), rng.normal(size=(6, 3))
    sums, _, _ = layers.embedding_grad(tokens, g, 5, 0.5)
    for v in range(5):
        for c in range(3):
            d = np.zeros_like(w)
            d[v, c] = 0.125
            up, down = (float(np.sum(layers.embedding(tokens, w + s * d, 0.5) * g)) for s in (1, -1))
            assert abs((up - down) / 0.25 - sums[v, c]) < 1e-13
