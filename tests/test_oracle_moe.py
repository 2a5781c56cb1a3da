"""Pins of the mixture-of-experts oracle: small cases by hand, gradients against
differences."""

import numpy as np
import pytest

from oracle import gemm, moe


def test_sort_by_hand():
    expert = np.array([[2, 0], [0, 7], [2, -1], [0, 2]])
    row, source, end = moe.sort(expert, 4, 1, 8)
    assert end.tolist() == [3, 3, 6, 6]
    assert row.tolist() == [[3, 0], [1, -1], [4, -1], [2, 5]]
    assert source.tolist() == [1, 2, 6, 0, 4, 7, -1, -1]
    row, source, end = moe.sort(expert, 4, 4, 16)
    assert end.tolist() == [4, 4, 8, 8]
    assert source.tolist() == [1, 2, 6, -1, 0, 4, 7, -1] + [-1] * 8


@pytest.mark.parametrize("tokens, topk, experts, align", [(1, 1, 1, 128), (3, 2, 4, 4), (5, 2, 3, 3), (2, 3, 8, 2)])
def test_rows_bound_is_the_most(tokens, topk, experts, align):
    rng = np.random.default_rng(0)
    most = 0
    for _ in range(400):
        e = rng.integers(0, experts, (tokens, topk)) if rng.random() < 0.7 else np.minimum(
            np.arange(tokens * topk).reshape(tokens, topk), rng.integers(0, experts, ()))
        most = max(most, moe.sort(e, experts, align, moe.rows_bound(tokens, topk, experts, align))[2][-1])
    assert most == moe.rows_bound(tokens, topk, experts, align)


def test_gather_and_combine_are_each_others_gradient():
    rng = np.random.default_rng(1)
    expert = rng.integers(-1, 3, (6, 2))
    row, source, _ = moe.sort(expert, 3, 2, 20)
    x, w, y = rng.normal(size=(6, 5)), rng.normal(size=(6, 2)), rng.normal(size=(20, 5))
    dout = rng.normal(size=(6, 5))
    # <combine(y), dout> is linear in y and in w
    out, _ = moe.combine(y, row, w)
    assert np.isclose((out * dout).sum(), (moe.gather(dout, source, 2, w) * y).sum())
    assert np.isclose((out * dout).sum(), (moe.combine_dweight(dout, y, row)[0] * w).sum())
    # <gather(x), y> = <x, combine(y)>
    assert np.isclose((moe.gather(x, source, 2) * y).sum(), (moe.combine(y, row)[0] * x).sum())


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(2)
    h, dy = rng.normal(size=(3, 8)) * 2, rng.normal(size=(3, 4))
    grad, size = moe.swiglu_grad(dy, h)
    assert (np.abs(grad) <= size + 1e-15).all()
    step = 1e-6
    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = step
        diff = ((moe.swiglu(h + d) - moe.swiglu(h - d)) * dy).sum() / (2 * step)
        assert abs(diff - grad[i]) < 1e-8
    assert moe.swiglu(np.array([[-800.0, 2.0]])).item() == 0.0
    assert moe.swiglu(np.array([[800.0, 2.0]])).item() == 1600.0


def test_grouped_wgrad_of_one_group_is_the_product():
    rng = np.random.default_rng(3)
    a, b = (rng.integers(0, 120, (4, 256)).astype(np.uint8) for _ in range(2))
    ra, rb = rng.random((4, 2)), rng.random((4, 2))
    want = gemm.blockwise_gemm(a, ra, b, rb, "1x128")
    out, _ = moe.grouped_wgrad(a, ra, b, rb, [0, 128, 128, 256])
    assert not out[0].any() and not out[2].any()
    assert np.allclose(out[1] + out[3], want)
