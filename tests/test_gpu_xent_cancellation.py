"""dH where rows of the head share a large component: a token's G sums to zero
over the vocabulary, so that component cancels, and only the rows' differences
reach dH.

Tolerances (u = 2^-24): dh[t] = sum_v G (w_v - w_target), G rounded to bf16 (at
most 2^-8 of it) and off by its logit's error dz = (K + 8) u sum|h w|, lse's
(2 dz + 2^-18 + 4 u |lse|) and its own exponential's, all relative to p; the
fp32 sums add (V + 8) u of the magnitudes summed, which hold the shared
component."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import metrics
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _f64(t):
    return t.detach().cpu().double().numpy()


def _case(T, V, K, shared, near, seed):
    """Rows of w: `shared` times their spread in common; tokens `near` their targets."""
    g = torch.Generator().manual_seed(seed)
    spread = 1.0 / K ** 0.5
    w = (torch.randn(V, K, generator=g) * spread + shared * spread * torch.randn(1, K, generator=g)).bfloat16()
    target = torch.randint(0, V, (T,), generator=g)
    h = (torch.randn(T, K, generator=g) * 0.25 + near * (w - w.float().mean(0)).float()[target]).bfloat16()
    return h, w, target, torch.randn(T, generator=g)


# 64-row tiles, shares of the contraction, 128-row tiles, 256 x 256 tiles with
# dH's contraction shared out, several pieces of the vocabulary
SHAPES = [(5, 300, 64), (40, 500, 1600), (100, 33000, 64), (300, 9000, 256), (1100, 4097, 192)]


@pytest.mark.parametrize("near", [0.0, 9.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_shared_component_cancels(gpu, shape, near):
    T, V, K = shape
    h, w, target, dloss = _case(T, V, K, 64.0, near, sum(shape))
    say("shared component", shape, near)
    args = [x.to(gpu) for x in (h, w, target)]
    _, lse = fp8.linear_xent_fwd(*args)
    dh, _ = fp8.linear_xent_bwd(dloss.to(gpu), *args, lse, need_dw=False)
    hf, wf, dl, t = _f64(h), _f64(w), _f64(dloss), np.arange(T)
    z = hf @ wf.T
    want_lse = z.max(axis=1) + np.log(np.exp(z - z.max(axis=1, keepdims=True)).sum(axis=1))
    p = np.exp(z - want_lse[:, None])
    g = p.copy()
    g[t, target.numpy()] = p[t, target.numpy()] - 1
    dz = (K + 8) * U * (np.abs(hf) @ np.abs(wf).T)
    rel = 2 * dz.max(axis=1) + dz.max(axis=1) + 2.0 ** -18 + 4 * U * np.abs(want_lse)
    got = _f64(dh)
    for i in t[:: max(1, T // 40)]:
        d = np.abs(wf - wf[target[i]])
        # of the target's own entry only the rounding of the others counts
        tol = abs(dl[i]) * ((2.0 ** -8 * np.abs(g[i]) + rel[i] * p[i]) @ d
                            + (V + 8) * U * (np.abs(g[i]) @ (np.abs(wf) + np.abs(wf[target[i]]))))
        want = dl[i] * (g[i] @ (wf - wf[target[i]]))
        err = np.abs(got[i] - want)
        assert np.all(err <= tol + metrics.bf16_ulp(np.abs(want) + tol) / 2 + 1e-37), (i, (err / tol).max())


# 128-row tiles, five pieces of the vocabulary, 64 x 256 tiles
@pytest.mark.parametrize("near", [0.0, 9.0])
@pytest.mark.parametrize("shape", [(100, 33000, 64), (8192, 40000, 64), (64, 131073, 64)])
def test_shared_component_cancels_over_many_columns(gpu, shape, near):
    """Where the worst case of the fp32 sums hides it: the error's rms, against
    that of independent roundings of G (2^-8 at most, each), of the output, and
    of fp32 sums that walk at random over V terms."""
    T, V, K = shape
    h, w, target, dloss = (x.to(gpu) for x in _case(T, V, K, 64.0, near, sum(shape)))
    say("shared component", shape, near)
    _, lse = fp8.linear_xent_fwd(h, w, target)
    dh, _ = fp8.linear_xent_bwd(dloss, h, w, target, lse, need_dw=False)
    hf, wf = h.double(), w.double()
    err = size = 0.0
    for i in range(0, T, 2048):
        rows = slice(i, i + 2048)
        z = hf[rows] @ wf.t()
        p = torch.softmax(z, 1)
        g = p.clone()
        g.scatter_add_(1, target[rows][:, None], torch.full_like(dloss[rows].double()[:, None], -1.0))
        dl = dloss[rows].double()[:, None]
        mean = wf.mean(0)
        d, own = wf - mean, (wf - mean)[target[rows]]
        want = dl * (g @ d)
        # sum_v g^2 (d_v - d_own)^2
        g2 = g.square()
        spread = g2 @ d.square() - 2 * own * (g2 @ d) + g2.sum(1, keepdim=True) * own.square()
        tol = dl.abs() * (2.0 ** -8 * spread.sqrt() + (V ** 0.5 + K) * U * (g.abs() @ wf.abs()))
        dz = (K ** 0.5 + 8) * U * (hf[rows].abs() @ wf.abs().t())        # of the logits, relative to p
        tol = tol + dl.abs() * ((p * dz) @ d.abs() + (p * dz).sum(1, keepdim=True) * own.abs())
        tol = tol + 2.0 ** -9 * want.abs()
        err += float((dh[rows].double() - want).square().sum())
        size += float(tol.square().sum())
    assert err <= size, (err / size) ** 0.5


def test_confident_tokens(gpu):
    """Tokens whose target has 1 - p of e^-9 or less of its probability, at
    logits of 1000: the others' entries of G and the target's, which lse alone
    gives only to 6e-5, still sum to zero."""
    T, V, K = 24, 300, 64
    g = torch.Generator().manual_seed(7)
    below = float(round(np.log(V)) + 9) + torch.randint(0, 3, (V,), generator=g).float()
    target = torch.arange(T) * 11
    h, w = torch.zeros(T, K), torch.zeros(V, K)
    h[:, 0], h[:, 1], w[:, 0], w[:, 1] = 1000.0, 1.0, 1.0, -below
    h[torch.arange(T), 8 + torch.arange(T)] = 1.0
    w[target, 8 + torch.arange(T)] = below[target]
    w[:, 40:] = torch.randn(V, 24, generator=g)           # no logit hangs on these
    h, w, dloss = h.bfloat16(), w.bfloat16(), torch.randn(T, generator=g) + 2.0
    say("shared component, confident tokens")
    args = [x.to(gpu) for x in (h, w, target)]
    _, lse = fp8.linear_xent_fwd(*args)
    dh, _ = fp8.linear_xent_bwd(dloss.to(gpu), *args, lse, need_dw=False)
    hf, wf, dl = _f64(h), _f64(w), _f64(dloss)
    z = hf @ wf.T
    for i in range(T):
        gap = z[i] - z[i, target[i]]
        p = np.exp(gap)
        p[target[i]] = 0.0
        p /= 1 + p.sum()
        d = wf - wf[target[i]]
        want, size = dl[i] * (p @ d), abs(dl[i]) * (p @ np.abs(d))
        # p to bf16; lse's rounding at 1000, and an exponential's at 40; the sums, which hold
        # the target's row times the others' total
        total = abs(dl[i]) * 2 * (p @ (np.abs(wf) + np.abs(wf[target[i]])))
        tol = (2.0 ** -8 + 2 * U * 1000 + 360 * U) * size + (V + 8) * U * total
        # the target's own entry, whatever it is, is summed and taken out again
        tol = tol + 4 * U * abs(dl[i]) * 2 * U * 1000 * np.abs(wf[target[i]])
        err = np.abs(_f64(dh)[i] - want)
        assert np.all(err <= tol + metrics.bf16_ulp(np.abs(want) + tol) / 2 + 1e-37), (i, (err / (tol + 1e-37)).max())
