"""Cross entropy of a linear head on the GPU against the 64-bit oracle.

Tolerances (u = 2^-24): a logit is K fp32 additions of exact products, within
dz = (K + 8) u sum|h w| of the exact one; lse and loss add the exponentials'
argument and value errors and the logarithm's, below 2^-18 + 4 u |lse|.  G is
off by its logit's and lse's error (relative), then rounded to bf16 (2^-8
relative: 8 significant bits); dh and dw add those through their products, one
rounding per term and half a bf16 spacing at the end."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import metrics, train
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IGNORE = -100


def _f64(t):
    return t.detach().cpu().double().numpy()


def _case(T, V, K, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, K, generator=g).bfloat16()
    w = (torch.randn(V, K, generator=g) * std / K ** 0.5).bfloat16()
    target = torch.randint(0, V, (T,), generator=g)
    dloss = torch.randn(T, generator=g)
    return h, w, target, dloss


def _close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(b[0] for b in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} off, first {i}: {got[i]!r} for {want[i]!r}, tol {np.broadcast_to(tol, got.shape)[i]!r}")


def _check(h, w, target, dloss, loss, lse, dh, dw, ignore=IGNORE):
    T, K = h.shape
    V = w.shape[0]
    hf, wf, dl = _f64(h), _f64(w), _f64(dloss)
    want_loss, want_lse, want_dh, want_dw = train.linear_xent(hf, wf, target.numpy(), ignore, dl)
    dz = (K + 8) * U * (np.abs(hf) @ np.abs(wf).T)
    tol = dz.max(axis=1) + 2.0 ** -18 + 4 * U * np.abs(want_lse)
    _close(_f64(lse), want_lse, tol, "lse")
    known = np.isfinite(want_loss)
    assert np.array_equal(np.isnan(_f64(loss)), ~known)
    _close(_f64(loss)[known], want_loss[known], 2 * tol[known], "loss")
    p = np.exp(hf @ wf.T - want_lse[:, None])
    counts = known & (target.numpy() != ignore)
    one = np.zeros_like(p)
    one[np.nonzero(counts)[0], target.numpy()[counts]] = 1.0
    weight = np.where(counts, np.abs(dl), 0.0)[:, None]
    size = np.abs(p - one) * weight
    g_tol = p * weight * (dz + tol[:, None]) + 2.0 ** -8 * size
    for got, want, t, what in (
            (dh, want_dh, g_tol @ np.abs(wf) + (V + 8) * U * (size @ np.abs(wf)), "dh"),
            (dw, want_dw, g_tol.T @ np.abs(hf) + (T + 8) * U * (size.T @ np.abs(hf)), "dw")):
        _close(_f64(got), want, t + metrics.bf16_ulp(np.abs(want) + t) / 2 + 1e-37, what)


# (T, V, K): one token, one column; below, on and past the tiles of 64 and 256;
# odd everything; large tiles (>= 128 of them, or with dH's splits); K of one
# slab and of an odd number of slabs
SHAPES = [(1, 1, 64), (1, 300, 64), (2, 7, 128), (63, 255, 192), (64, 256, 256), (65, 257, 320),
          (300, 511, 64), (129, 1000, 512), (256, 4099, 128), (2049, 4097, 192), (2048, 4096, 64),
          (300, 33001, 320), (1025, 7777, 256)]


@pytest.mark.parametrize("shape", SHAPES)
def test_forward_backward(gpu, shape):
    h, w, target, dloss = _case(*shape, seed=sum(shape))
    T = shape[0]
    target[torch.arange(T) % 5 == 3] = IGNORE
    say("linear_xent", shape)
    hd, wd, td = h.to(gpu), w.to(gpu), target.to(gpu)
    loss, lse = fp8.linear_xent_fwd(hd, wd, td, IGNORE)
    dh, dw = fp8.linear_xent_bwd(dloss.to(gpu), hd, wd, td, lse, IGNORE)
    torch.cuda.synchronize()
    _check(h, w, target, dloss, loss, lse, dh, dw)


@pytest.mark.parametrize("shape", [(1, 500, 1600), (3, 1001, 4096), (64, 4097, 1536), (70, 129, 2112), (1000, 65, 1600)])
def test_long_contractions_of_few_tiles(gpu, shape):
    """Logits whose contraction is shared out; with targets that do not count."""
    h, w, target, dloss = _case(*shape, seed=sum(shape))
    target[0 if shape[0] > 1 else 1:1] = shape[1] + 5
    target[2::5] = IGNORE
    args = [t.to(gpu) for t in (h, w, target)]
    say(f"linear_xent shares {shape}")
    loss, lse = fp8.linear_xent_fwd(*args)
    dh, dw = fp8.linear_xent_bwd(dloss.to(gpu), *args, lse)
    _check(h, w, target, dloss, loss, lse, dh, dw)
    again = fp8.linear_xent_bwd(dloss.to(gpu), *args, lse)
    assert torch.equal(fp8.linear_xent_fwd(*args)[1], lse) and torch.equal(again[0], dh) and torch.equal(again[1], dw)


def test_strided_operands_and_single_gradients(gpu):
    """Column slices of wider buffers; a gradient left out changes nothing."""
    T, V, K = 200, 1500, 192
    h, w, target, dloss = _case(T, V, K + 64, seed=4)
    hd, wd = h.to(gpu)[:, 32:32 + K], w.to(gpu)[:, 8:8 + K]
    td, dd = target.to(gpu), dloss.to(gpu)
    say("linear_xent strided")
    loss, lse = fp8.linear_xent_fwd(hd, wd, td)
    dh, dw = fp8.linear_xent_bwd(dd, hd, wd, td, lse)
    _check(hd.cpu(), wd.cpu(), target, dloss, loss, lse, dh, dw)
    only_h = fp8.linear_xent_bwd(dd, hd, wd, td, lse, need_dw=False)
    only_w = fp8.linear_xent_bwd(dd, hd, wd, td, lse, need_dh=False)
    assert only_h[1] is None and torch.equal(only_h[0], dh)
    assert only_w[0] is None and torch.equal(only_w[1], dw)
    assert fp8.linear_xent_bwd(dd, hd, wd, td, lse, need_dh=False, need_dw=False) == (None, None)


@pytest.mark.parametrize("shape", [(40, 700, 256), (100, 20000, 512), (700, 9000, 1024), (2049, 4097, 192)])
def test_gradients_together_and_alone(gpu, shape):
    """Both gradients in one launch, or in two where their tiles differ, have
    the bits of each by itself."""
    h, w, target, dloss = (t.to(gpu) for t in _case(*shape, seed=sum(shape)))
    say(f"linear_xent gradients {shape}")
    _, lse = fp8.linear_xent_fwd(h, w, target)
    dh, dw = fp8.linear_xent_bwd(dloss, h, w, target, lse)
    assert torch.equal(dh, fp8.linear_xent_bwd(dloss, h, w, target, lse, need_dw=False)[0])
    assert torch.equal(dw, fp8.linear_xent_bwd(dloss, h, w, target, lse, need_dh=False)[1])


def test_targets_that_do_not_count(gpu):
    """Ignored tokens (another ignore_index, in the vocabulary too), targets
    outside it, and weights of zero: no gradient, whatever the token holds."""
    T, V, K = 70, 600, 128
    h, w, target, dloss = _case(T, V, K, seed=5)
    target[:10], target[10], target[11], target[12] = 17, -1, V, V + 10 ** 9
    dloss[20:25] = 0.0
    say("linear_xent uncounted targets")
    args = [t.to(gpu) for t in (h, w, target)]
    loss, lse = fp8.linear_xent_fwd(*args, ignore_index=17)
    dh, dw = fp8.linear_xent_bwd(dloss.to(gpu), *args, lse, ignore_index=17)
    _check(h, w, target, dloss, loss, lse, dh, dw, ignore=17)
    assert not loss[:10].any() and bool(loss[10:13].isnan().all())
    assert not dh[:13].any() and not dh[20:25].any()
    # every token ignored: zero losses and gradients
    none = torch.full((T,), 17, device=gpu)
    loss, lse = fp8.linear_xent_fwd(args[0], args[1], none, ignore_index=17)
    dh, dw = fp8.linear_xent_bwd(dloss.to(gpu), args[0], args[1], none, lse, ignore_index=17)
    assert not loss.any() and not dh.any() and not dw.any() and bool(lse.isfinite().all())


def test_masked_token_with_infinities(gpu):
    """An ignored token's own values do not reach its loss or gradient, nor
    any other token's."""
    T, V, K = 40, 500, 64
    h, w, target, dloss = _case(T, V, K, seed=6)
    target[7] = IGNORE
    bad = h.clone()
    bad[7, 3], bad[7, 5] = float("inf"), float("nan")
    args = [t.to(gpu) for t in (w, target)]
    say("linear_xent masked infinities")
    good = fp8.linear_xent_fwd(h.to(gpu), *args)
    loss, lse = fp8.linear_xent_fwd(bad.to(gpu), *args)
    others = torch.arange(T) != 7
    assert loss[7] == 0 and torch.equal(loss, good[0]) and torch.equal(lse[others.to(gpu)], good[1][others.to(gpu)])
    dh, _ = fp8.linear_xent_bwd(dloss.to(gpu), bad.to(gpu), *args, lse, need_dw=False)
    want, _ = fp8.linear_xent_bwd(dloss.to(gpu), h.to(gpu), *args, good[1], need_dw=False)
    assert not dh[7].any() and torch.equal(dh, want)


@pytest.mark.parametrize("shape", [(40, 500, 64), (40, 500, 1600), (130, 1000, 192), (1025, 7777, 256)])
def test_masked_infinities_stay_out_of_dw(gpu, shape):
    """Infinities and NaN in tokens that have no gradient (ignored, outside the
    vocabulary, weight 0), the last one among them: dw and dh are those of
    finite values there."""
    T, V, K = shape
    h, w, target, dloss = _case(T, V, K, seed=16)
    target[7], target[T - 1], target[33], dloss[21] = IGNORE, IGNORE, V + 3, 0.0
    bad = h.clone()
    bad[7, 3], bad[T - 1, 0], bad[33, 5], bad[21, K - 1] = float("inf"), float("nan"), float("-inf"), float("nan")
    w, target, dloss = (t.to(gpu) for t in (w, target, dloss))
    say(f"linear_xent masked infinities {shape}")
    grads = []
    for x in (h.to(gpu), bad.to(gpu)):
        lse = fp8.linear_xent_fwd(x, w, target)[1]
        grads.append(fp8.linear_xent_bwd(dloss, x, w, target, lse))
    for got, want in zip(grads[1], grads[0]):
        assert torch.equal(got, want)


def test_large_logits(gpu):
    """Logits of thousands: the maximum is taken out before the exponential."""
    T, V, K = 66, 777, 64
    h, w, target, dloss = _case(T, V, K, seed=8, std=2.0)
    h, w = h * 64, w * 16
    say("linear_xent large logits")
    args = [t.to(gpu) for t in (h, w, target)]
    loss, lse = fp8.linear_xent_fwd(*args)
    dh, dw = fp8.linear_xent_bwd(dloss.to(gpu), *args, lse)
    assert bool(loss.isfinite().all()) and bool(dh.isfinite().all()) and bool(dw.isfinite().all())
    _check(h, w, target, dloss, loss, lse, dh, dw)


def test_repeats_and_empty(gpu):
    T, V, K = 1500, 9001, 128
    h, w, target, dloss = (t.to(gpu) for t in _case(T, V, K, seed=9))
    say("linear_xent repeats")
    loss, lse = fp8.linear_xent_fwd(h, w, target)
    grads = fp8.linear_xent_bwd(dloss, h, w, target, lse)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip((loss, lse), fp8.linear_xent_fwd(h, w, target)))
        assert all(torch.equal(a, b) for a, b in zip(grads, fp8.linear_xent_bwd(dloss, h, w, target, lse)))
    e = fp8.linear_xent_fwd(h[:0], w, target[:0])
    assert e[0].shape == (0,) and e[1].shape == (0,)
    dh, dw = fp8.linear_xent_bwd(dloss[:0], h[:0], w, target[:0], e[1])
    assert dh.shape == (0, K) and dw.shape == (V, K) and not dw.any()


def test_vocabulary_in_several_pieces(gpu):
    """A vocabulary of several workspace pieces equals the same call on rows
    of it (dH adds over the pieces; dW's rows are each one piece's)."""
    T, V, K = 8192, 40000, 64
    h, w, target, dloss = (t.to(gpu) for t in _case(T, V, K, seed=10))
    say("linear_xent pieces")
    loss, lse = fp8.linear_xent_fwd(h, w, target)
    dh, dw = fp8.linear_xent_bwd(dloss, h, w, target, lse)
    z = h.double() @ w.double().t()
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    assert float((lse.double() - torch.logsumexp(z, 1)).abs().max()) < 1e-4
    p[torch.arange(T, device=gpu), target] -= 1
    p *= dloss.double()[:, None]
    for got, want in ((dh, p @ w.double()), (dw, p.t().contiguous() @ h.double())):
        # two roundings to bf16 (G's and the output's), 2^-8 each at most
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -7
