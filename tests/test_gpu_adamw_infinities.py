"""AdamW and gradients that are infinite or NaN.  8-bit states: the element itself is
lost (NaN from then on, as its fp32 states would be), its block's other
elements are not."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import e4m3
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

N = 1000
BAD = {5: float("inf"), 200: float("-inf"), 400: float("nan"), 999: float("inf")}


def _state(gpu):
    return [torch.zeros(N, dtype=torch.uint8, device=gpu) for _ in range(2)] + [torch.ones(8, device=gpu) for _ in range(2)]


def _step(p, g, s, step, seed):
    fp8.adamw_step([p], [g], [s[0]], [s[1]], exp_avg_scales=[s[2]], root_scales=[s[3]], step=step, lr=1e-2,
                   seed=None if seed is None else seed + step)


@pytest.mark.parametrize("seed", [None, 17])
def test_neighbours_of_infinities(gpu, seed):
    g = torch.Generator().manual_seed(2)
    grads = [(torch.randn(N, generator=g) * 1e-3) for _ in range(3)]
    start = torch.randn(N, generator=g)
    kept = torch.ones(N, dtype=torch.bool)
    kept[list(BAD)] = False
    runs = []
    for bad in (False, True):
        p, s = start.to(gpu), _state(gpu)
        say("adamw infinities", seed, bad)
        for step, grad in enumerate(grads, 1):
            d = grad.clone()
            d[~kept] = 0.0                     # the same blocks without these elements
            if bad and step == 1:
                for i, x in BAD.items():
                    d[i] = x
            _step(p, d.to(gpu), s, step, seed)
        runs.append([t.cpu() for t in (p, *s)])
    clean, got = runs
    for a, b in zip(clean[:3], got[:3]):       # parameters and codes
        assert torch.equal(a[kept], b[kept])
    assert torch.equal(clean[3], got[3]) and torch.equal(clean[4], got[4])
    decoded = [e4m3.decode(t.numpy()) for t in got[1:3]]
    for i in BAD:
        assert bool(got[0][i].isnan()) and np.isnan(decoded[0][i]) and np.isnan(decoded[1][i]), i


@pytest.mark.parametrize("seed", [None, 17])
def test_a_square_past_fp32(gpu, seed):
    """1e30 has a first moment, on whose scale its block's are held, and no
    second one: its root is NaN, the block's other roots are untouched."""
    g = torch.Generator().manual_seed(4)
    d = torch.randn(N, generator=g) * 1e-3
    roots = []
    say("adamw square past fp32", seed)
    for x in (0.0, 1e30):
        d[7] = x
        p, s = torch.zeros(N, device=gpu), _state(gpu)
        _step(p, d.to(gpu), s, 1, seed)
        roots.append((s[1].cpu(), s[3].cpu()))
    others = torch.arange(N) != 7
    assert torch.equal(roots[0][0][others], roots[1][0][others]) and torch.equal(roots[0][1], roots[1][1])
    assert np.isnan(e4m3.decode(roots[1][0].numpy())[7]) and bool(s[2].isfinite().all())
    assert abs(float(e4m3.decode(s[0].cpu().numpy())[7]) * float(s[2][0]) / 1e29 - 1) < 0.13


@pytest.mark.parametrize("seed", [None, 17])
def test_finite_extremes(gpu, seed):
    """The largest first moments that exist keep finite codes."""
    p, s = torch.zeros(N, device=gpu), _state(gpu)
    d = torch.full((N,), 1e18, device=gpu)     # squares near 1e36
    say("adamw extremes", seed)
    _step(p, d, s, 1, seed)
    assert bool(p.isfinite().all())
    m = e4m3.decode(s[0].cpu().numpy()) * np.repeat(s[2].cpu().double().numpy(), 128)[:N]
    r = e4m3.decode(s[1].cpu().numpy()) * np.repeat(s[3].cpu().double().numpy(), 128)[:N]
    assert np.all(np.abs(m / 1e17 - 1) < 0.13) and np.all(np.abs(r / (1e18 * np.sqrt(1e-3)) - 1) < 0.13)


@pytest.mark.parametrize("seed", [None, 17])
def test_a_nan_moment_stays_one(gpu, seed):
    """A NaN code in either state alone, as a checkpoint may hold one."""
    d = torch.randn(N, generator=torch.Generator().manual_seed(6)) * 1e-3
    for which in (0, 1):
        p, s = torch.zeros(N, device=gpu), _state(gpu)
        s[which][300] = 0x7F
        s[which][301] = 0xFF
        say("adamw nan codes", seed, which)
        for step in (1, 2):
            _step(p, d.to(gpu), s, step, seed)
            bad = np.isnan(e4m3.decode(s[which].cpu().numpy()))
            assert bad[300] and bad[301] and bad.sum() == 2
        assert int(p.isnan().sum()) == 2 and bool(p[300:302].isnan().all())
        assert bool(s[2].isfinite().all()) and bool(s[3].isfinite().all())
def test_nan_stays_nan_in_bf16_parameters(gpu):
    """A NaN with every mantissa bit set does not carry into the sign."""
    n = 256
    for bits in (8, 32):
        p = torch.ones(n, device=gpu).bfloat16()
        grad = torch.full((n,), -1, dtype=torch.int32, device=gpu).view(torch.float32)
        m, v = (torch.zeros(n, dtype=torch.uint8 if bits == 8 else torch.float32, device=gpu) for _ in range(2))
        s = [torch.ones(2, device=gpu) for _ in range(2)] if bits == 8 else None
        say("adamw nan", bits)
        fp8.adamw_step([p], [grad], [m], [v], exp_avg_scales=s and [s[0]], root_scales=s and [s[1]], step=1, lr=0.1, seed=3)
        assert bool(p.isnan().all()), (bits, p[:8])
