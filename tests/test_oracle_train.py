"""The 64-bit oracle of the norm, cross entropy and AdamW: gradients against
central differences, closed forms, and the random rounding's mean."""

import numpy as np
import pytest

from oracle import e4m3, train

RNG = np.random.default_rng


def _differences(f, x, step=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        out[i] = (f(hi) - f(lo)) / (2 * step)
    return out


@pytest.mark.parametrize("with_dres", [False, True])
def test_norm_gradients_are_the_differences(with_dres):
    rng = RNG(1)
    s, w, dy = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7))
    dres = rng.normal(size=(3, 7)) if with_dres else None

    def value(s_, w_):
        v = (dy * train.rms_norm_fwd(s_, w_, 1e-3)[0]).sum()
        return v + (0 if dres is None else (dres * s_).sum())
    dx, dw = train.rms_norm_bwd(dy, s, w, 1e-3, dres)
    # central differences: error step^2 f''' / 6 + rounding 1e-16 / step, below 1e-8
    assert np.abs(dx - _differences(lambda a: value(a, w), s)).max() < 1e-8
    assert np.abs(dw - _differences(lambda a: value(s, a), w)).max() < 1e-8


def test_norm_closed_forms():
    v, rstd = train.rms_norm_fwd(np.full((2, 16), 3.0), np.ones(16), 0.0)
    assert np.allclose(v, 1.0) and np.allclose(rstd, 1 / 3)
    v, rstd = train.rms_norm_fwd(np.zeros((1, 16)), np.ones(16), 1e-4)
    assert not v.any() and np.allclose(rstd, 100.0)


def test_xent_gradients_are_the_differences():
    rng = RNG(2)
    h, w = rng.normal(size=(5, 4)), rng.normal(size=(9, 4))
    target, dl = np.array([0, 8, -100, 3, 3]), np.array([1.0, -2.0, 5.0, 0.0, 0.25])

    def value(h_, w_):
        return (train.linear_xent(h_, w_, target)[0] * dl).sum()
    _, _, dh, dw = train.linear_xent(h, w, target, dloss=dl)
    assert np.abs(dh - _differences(lambda a: value(a, w), h)).max() < 1e-8
    assert np.abs(dw - _differences(lambda a: value(h, a), w)).max() < 1e-8
    assert not dh[2].any() and not dh[3].any()


def test_xent_closed_forms():
    loss, lse = train.linear_xent(np.zeros((2, 4)), np.ones((10, 4)), np.array([3, -100]))
    assert np.allclose(lse, np.log(10)) and np.allclose(loss, [np.log(10), 0])
    loss, _ = train.linear_xent(np.zeros((1, 4)), np.ones((10, 4)), np.array([10]))
    assert np.isnan(loss[0])


def test_adamw_first_step_is_a_signed_step():
    """From zero states the first step is lr sign(g) (eps aside) plus decay."""
    g, p = np.array([3.0, -1e-3, 0.0]), np.array([1.0, 2.0, 4.0])
    q, m, v = train.adamw(p, g, 0 * p, 0 * p, step=1, lr=0.1, beta1=0.9, beta2=0.99, eps=0.0 + 1e-30,
                          weight_decay=0.5)
    assert np.allclose(q, p - 0.1 * np.sign(g) - 0.05 * p)
    assert np.allclose(m, 0.1 * g) and np.allclose(v, 0.01 * g * g)


def test_state_scales_are_the_least_power_of_two():
    x = np.zeros(128 * 4 + 5)
    x[0], x[128], x[256], x[-1] = 448.0, -448.0001, 1e-30, 1.0
    s = train.state_scales(x)
    assert s[0] == 1 and s[1] == 2 and s[3] == 1
    for k, top in ((2, 1e-30), (4, 1.0)):
        assert top <= 448 * s[k] < 2 * top * 1.0000001 or top > 448 * s[k] / 2


def test_neighbours_are_the_grid():
    """Every E4M3 value is its own neighbour; between two it gives both."""
    grid = np.array(sorted({abs(float(x)) for x in e4m3.decode(np.arange(127, dtype=np.uint8))}))
    down, up, _ = train.e4m3_neighbours(grid)
    assert np.array_equal(down, grid) and np.array_equal(up, grid)
    mid = (grid[1:] + grid[:-1]) / 2
    down, up, _ = train.e4m3_neighbours(mid)
    assert np.array_equal(down, grid[:-1]) and np.array_equal(up, grid[1:])


def test_random_rounding_has_the_values_mean():
    """Mean of 65536 roundings with every 16-bit number: the value, to 2^-16 of the spacing."""
    r = np.arange(65536)
    for y in (1.03, -300.7, 0.0077, 2.0 ** -11, 447.9):
        _, _, ulp = train.e4m3_neighbours(np.array([y]))
        assert abs(train.e4m3_stochastic(np.full(65536, y), r).mean() - y) <= ulp[0] * 2.0 ** -16


def test_random_bits_are_even_and_unrelated():
    n = 1 << 18
    streams = [b.astype(np.float64) / 65536 for b in train.random_bits(12345678901234567, 3, n)]
    streams.append(train.random_bits(12345678901234568, 3, n)[0] / 65536.0)
    streams.append(train.random_bits(12345678901234567, 4, n)[0] / 65536.0)
    tol = 5 / np.sqrt(n)      # five standard errors of a mean of n values of variance <= 1
    for a in streams:
        assert abs(a.mean() - 0.5) < tol * np.sqrt(1 / 12) and abs(a.var() * 12 - 1) < tol
        assert abs(np.corrcoef(a[:-1], a[1:])[0, 1]) < tol and abs(np.corrcoef(a[:-128], a[128:])[0, 1]) < tol
    for i, a in enumerate(streams):
        for b in streams[i + 1:]:
            assert abs(np.corrcoef(a, b)[0, 1]) < tol
