"""Cross entropy of tokens whose target has almost all of the probability:
1 - p of 1e-6 to 1e-4 at logits of 20, 100 and 1000.  The loss is about 1 - p,
and so is the target's entry of G, both far below a rounding of the logits.

Every logit is a sum of few numbers that fp32 holds exactly, so all error is
the operator's own.  Tolerances (u = 2^-24), relative: an exponential's
argument d is rounded in its product with log2 e and by that constant (2 u d),
the sum of exponentials by its terms (at most 128 in sequence or by levels), d
itself by u d and the logarithm's 2 u d, the functions by a few u: REL = (5 d +
160) u at d = 40.  G is rounded to bf16, half a spacing of which is at most
2^-8 of it, and dw adds fp32 sums (T terms) and half a spacing."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import metrics
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
REL = (5 * 40 + 160) * U
LEVELS = (20.0, 100.0, 1000.0)


def _case(T, V, K, seed):
    """z[t, target] = level(t); the other columns' logits lie ln(V) + 9 to
    ln(V) + 18 below it: 1 - p is about e^-18 to e^-9."""
    g = torch.Generator().manual_seed(seed)
    targets = min(32, V // 4)
    rows = torch.randperm(V, generator=g)[:targets]
    below = float(round(np.log(V)) + 9) + torch.randint(0, 3, (V,), generator=g).float()
    part = torch.randint(0, 256, (V,), generator=g).float() / 256
    part[rows] = 0.0
    w, h = torch.zeros(V, K), torch.zeros(T, K)
    t = torch.arange(T)
    h[:, 0], h[:, 1], h[:, 2] = torch.tensor(LEVELS)[t % 3], 1.0, 1.0
    w[:, 0], w[:, 1], w[:, 2] = 1.0, -below, -part
    group = t % targets
    h[t, 3 + group] = 1.0
    w[rows, 3 + torch.arange(targets)] = below[rows]      # cancels it for the group's own tokens
    h[:, 40] = -2.25 * (t % 4).float()                    # the other columns further down
    w[:, 40] = 1.0
    w[rows, 40] = 0.0
    return h.bfloat16(), w.bfloat16(), rows[group], torch.randn(T, generator=g) + 2.0


# few and many tokens: 64-row tiles, shares of the contraction, 128-row tiles,
# 256 x 256 tiles, 64 x 256 tiles
SHAPES = [(9, 300, 64), (9, 300, 1600), (100, 33000, 64), (300, 33001, 64), (33, 131073, 64)]


@pytest.mark.parametrize("shape", SHAPES)
def test_confident_tokens(gpu, shape):
    h, w, target, dloss = _case(*shape, seed=sum(shape))
    T, V, K = shape
    say("confident tokens", shape)
    b = w.to(gpu).requires_grad_()
    loss = fp8.linear_cross_entropy(h.to(gpu), b, target.to(gpu), reduction="none")
    loss.backward(dloss.to(gpu))
    torch.cuda.synchronize()
    hf, wf, dl = (x.double().numpy() for x in (h, w, dloss))
    z = hf @ wf.T
    t = np.arange(T)
    gap = z - z[t, target.numpy()][:, None]
    gap[t, target.numpy()] = -np.inf
    rest = np.exp(gap).sum(axis=1)                        # (1 - p) / p
    want = np.log1p(rest)
    assert 1e-9 < want.min() and want.max() < 1e-3 and -gap[np.isfinite(gap)].max() < 40
    got = loss.detach().cpu().double().numpy()
    assert np.all(np.abs(got - want) <= REL * want), (np.abs(got / want - 1).max(), REL)
    g = np.exp(gap) / (1 + rest)[:, None]
    g[t, target.numpy()] = -rest / (1 + rest)
    g *= dl[:, None]
    size = np.abs(g).T @ np.abs(hf)
    # lse itself is one fp32 number: the other columns share its rounding
    lse_tol = 2 * U * np.abs(z).max()
    tol = (2.0 ** -8 + REL + lse_tol + (T + 8) * U) * size
    want = g.T @ hf
    bad = np.abs(b.grad.cpu().double().numpy() - want) > tol + metrics.bf16_ulp(np.abs(want) + tol) / 2
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])


def test_confident_tokens_without_the_losses(gpu):
    """The backward from lse alone: the target's entry is off by lse's own
    rounding, and nothing else is."""
    h, w, target, dloss = _case(9, 300, 64, seed=1)
    args = [x.to(gpu) for x in (h, w, target)]
    say("confident tokens, lse alone")
    loss, lse = fp8.linear_xent_fwd(*args)
    _, dw = fp8.linear_xent_bwd(dloss.to(gpu), *args, lse)
    _, want = fp8.linear_xent_bwd(dloss.to(gpu), *args, lse, loss=loss)
    off = (dw.double() - want.double()).abs().cpu().numpy()
    tol = (8 * U * np.abs(h.double().numpy()[:, :1]) + 2.0 ** -7 * loss.cpu().double().numpy()[:, None]) * np.abs(dloss.double().numpy())[:, None]
    assert np.all(off <= tol.sum() * np.abs(h.double().numpy()).max(axis=0) + metrics.bf16_ulp(np.abs(want.double().cpu().numpy())))
    assert bool((dw[:, 1] != want[:, 1]).any())


def test_one_column_and_columns_that_vanish(gpu):
    """A vocabulary of one column has loss 0 and no gradient; columns at -inf
    leave the target alone with all of the probability."""
    say("one column")
    h = torch.ones(3, 64, device=gpu).bfloat16()
    for V in (1, 5, 200):
        w = torch.full((V, 64), float("-inf"), device=gpu).bfloat16()
        w[0] = 0.25
        target = torch.zeros(3, dtype=torch.int64, device=gpu)
        loss, lse = fp8.linear_xent_fwd(h, w, target)
        assert not loss.any() and bool((lse == 16.0).all())
        if V == 1:
            dh, dw = fp8.linear_xent_bwd(torch.ones(3, device=gpu), h, w, target, lse, loss=loss)
            assert not dh.any() and not dw.any()
        else:
            loss, lse = fp8.linear_xent_fwd(h, w, target + 1)
            assert bool((loss == float("inf")).all()) and bool((lse == 16.0).all())


def test_losses_changed_in_place(gpu):
    """What a caller does to the losses does not reach the backward's softmax."""
    h, w, target, dloss = (x.to(gpu) for x in _case(9, 300, 64, seed=2))
    grads = []
    say("losses in place")
    for change in (False, True):
        a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
        loss = fp8.linear_cross_entropy(a, b, target, reduction="none")
        if change:
            loss *= 2.0
            loss.backward(dloss / 2)
        else:
            loss.backward(dloss)
        grads.append((a.grad, b.grad))
    assert all(torch.equal(x, y) for x, y in zip(*grads))
