"""The token operators' oracle against what defines it: differences, inverses, the format's own bounds."""
import numpy as np
import pytest

from oracle import token_oracle as o


def test_layer_norm_rows_are_normalised():
    x = np.random.default_rng(0).normal(3.0, 2.0, (5, 33))
    y, mean, rstd, xh = o.layer_norm(x, eps=1e-12)
    assert np.allclose(y, xh) and np.allclose(xh.mean(1), 0, atol=1e-14) and np.allclose((xh ** 2).mean(1), 1)
    assert np.allclose(mean, x.mean(1)) and np.allclose(rstd, 1 / x.std(1))
    w, b = np.arange(33.0), np.ones(33)
    assert np.allclose(o.layer_norm(x, w, b, 1e-12)[0], xh * w + 1)


@pytest.mark.parametrize("D", [1, 2, 17])
def test_layer_norm_backward_against_differences(D):
    rng = np.random.default_rng(D)
    x, dy, w, b = rng.normal(size=(4, D)), rng.normal(size=(4, D)), rng.normal(size=D), rng.normal(size=D)
    eps, h = 1e-2, 1e-6
    _, _, rstd, xh = o.layer_norm(x, w, b, eps)
    dx, dw, db = o.layer_norm_backward(dy, xh, rstd, w)
    loss = lambda x, w, b: (dy * o.layer_norm(x, w, b, eps)[0]).sum()  # noqa: E731
    for i in range(4):
        for j in range(D):
            d = np.zeros_like(x)
            d[i, j] = h
            assert abs((loss(x + d, w, b) - loss(x - d, w, b)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(D):
        d = np.zeros(D)
        d[j] = h
        assert abs((loss(x, w + d, b) - loss(x, w - d, b)) / (2 * h) - dw[j]) < 1e-7
        assert abs((loss(x, w, b + d) - loss(x, w, b - d)) / (2 * h) - db[j]) < 1e-7


def test_rope_grid_order():
    g = o.rope_grid(2, 3, 4, pos0=(10.0, 0.0, -1.0), step=(1.0, 2.0, 0.5))
    assert np.array_equal(g[(1 * 3 + 2) * 4 + 3], [11.0, 4.0, 0.5])


@pytest.mark.parametrize("halves", [False, True])
def test_rope_turns(halves):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(6, 2, 14))
    pos = rng.integers(0, 50, (6, 3)).astype(float)
    axes = (4, 2, 6)
    y = o.rope(x, pos, axes, theta=100.0, halves=halves)
    assert np.array_equal(y[..., 12:], x[..., 12:])                         # the rest is copied
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(o.rope(y, pos, axes, 100.0, halves, inverse=True), x)
    assert np.array_equal(o.rope(x, 0 * pos, axes, 100.0, halves), x)
    # pair 1 of the width axis is pair 4 of all: by hand
    a, b = (4, 10) if halves else (8, 9)
    ang = pos[:, 2] * 100.0 ** (-2 / 6)
    assert np.allclose(y[:, 0, a], x[:, 0, a] * np.cos(ang) - x[:, 0, b] * np.sin(ang))
    assert np.allclose(y[:, 0, b], x[:, 0, a] * np.sin(ang) + x[:, 0, b] * np.cos(ang))
    # scores depend on differences of positions only
    z = rng.normal(size=(6, 2, 14))
    s0 = (y * o.rope(z, pos, axes, 100.0, halves)).sum(-1)
    s1 = (o.rope(x, pos + 7, axes, 100.0, halves) * o.rope(z, pos + 7, axes, 100.0, halves)).sum(-1)
    assert np.allclose(s0, s1)


def test_rope_gradient_is_the_transpose():
    rng = np.random.default_rng(4)
    x, dy = rng.normal(size=(3, 2, 8)), rng.normal(size=(3, 2, 8))
    pos = rng.normal(size=(3, 3)) * 10
    dx = o.rope(dy, pos, (2, 2, 4), inverse=True)
    h = 1e-6
    v = rng.normal(size=x.shape)
    f = lambda t: (dy * o.rope(x + t * v, pos, (2, 2, 4))).sum()  # noqa: E731
    assert abs((f(h) - f(-h)) / (2 * h) - (dx * v).sum()) < 1e-7


def test_checkpoint_bounds_and_exact_values():
    rng = np.random.default_rng(5)
    x = (rng.normal(size=(40, 75)) * np.exp(3 * rng.normal(size=(40, 1)))).astype(np.float32).astype(np.float64)
    codes, scales = o.checkpoint(x)
    v = o.checkpoint_values(codes, scales)
    e = np.repeat(scales.astype(float) - 127, 32, axis=1)[:, :75]
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (e - 10)))
    for j in range(3):
        top = np.abs(x[:, 32 * j: 32 * j + 32]).max(1)
        s = 2.0 ** (scales[:, j].astype(float) - 127)
        assert np.all(top <= 448 * s) and np.all(top > 224 * s)
    again = o.checkpoint(v)                                                 # what it stands for stays
    assert np.array_equal(o.checkpoint_values(*again), v)


def test_checkpoint_ties_and_edges():
    one = np.zeros((1, 32))
    one[0, :6] = [448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -10]
    codes, scales = o.checkpoint(one)
    assert scales[0, 0] == 127
    assert np.array_equal(o.checkpoint_values(codes, scales)[0, :6], [448.0, 16.0, 20.0, 0.0, 2.0 ** -8, 0.0])
    big = np.full((1, 33), np.finfo(np.float32).max, dtype=np.float64)
    big[0, 1:4] = [np.nan, np.inf, -np.inf]
    big[0, 32] = 0.0
    codes, scales = o.checkpoint(big)
    v = o.checkpoint_values(codes, scales)
    assert list(scales[0]) == [247, 0] and v[0, 0] == 240.0 * 2.0 ** 120 and v[0, 32] == 0
    assert np.all(np.isnan(v[0, 1:4])) and np.all(np.isfinite(v[0, 4:]))
