"""Modules of the training step: frozen parts, inputs of any layout, autograd's
record of what was changed in place, checkpoints of other settings, the loss in
a graph."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from blockwise_scaled_fp8_amd import ops
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _randn(gpu, *shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).bfloat16().to(gpu)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("frozen", ["weight", "rest", "norm", "input"])
def test_norm_linear_with_frozen_parts(gpu, monkeypatch, frozen, residual):
    """Frozen parts cost no product and no codes; the other gradients keep
    their bits."""
    M, K, N = 256, 384, 512
    m = fp8.RMSNormLinear(K, N, device=gpu)
    x, r, dy = _randn(gpu, M, K, seed=1), _randn(gpu, M, K, seed=2), _randn(gpu, M, N, seed=3)
    products, norms = [], []
    gemm, norm = ops.fp8_scaled_gemm_blockwise, ops.rms_norm_fwd

    def counted(*a, **k):
        products.append(1)
        return gemm(*a, **k)

    def watched(*a, **k):
        norms.append(k["qt"])
        return norm(*a, **k)
    monkeypatch.setattr(ops, "fp8_scaled_gemm_blockwise", counted)
    monkeypatch.setattr(ops, "rms_norm_fwd", watched)
    grads = []
    say("RMSNormLinear frozen", frozen)
    for freeze in (False, True):
        m.norm.weight.requires_grad_(not freeze or frozen in ("weight", "input"))
        m.linear.weight.requires_grad_(not freeze or frozen != "weight")
        a, b = (t.clone().requires_grad_(not freeze or frozen in ("weight", "norm")) for t in (x, r))
        m.zero_grad(set_to_none=True)
        products.clear()
        norms.clear()
        y = m(a, b)[0] if residual else m(a)
        y.backward(dy)
        grads.append([t.grad for t in (a, b, m.norm.weight, m.linear.weight)])
        # forward, data gradient, weight gradient
        want = 3 if not freeze or frozen in ("norm", "input") else 2
        assert len(products) == want and norms == [not (freeze and frozen == "weight")]
    for full, part in zip(*grads):
        assert part is None or torch.equal(full, part)
    assert sum(t is not None for t in grads[1]) >= 1


def _layouts(t):
    """The same values expanded, transposed, off alignment, at an odd row pitch."""
    rows, cols = t.shape
    flat = torch.zeros(rows * cols + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    wide = torch.zeros(rows, cols + 5, dtype=t.dtype, device=t.device)
    wide[:, 3:3 + cols] = t
    return {"transposed": t.t().contiguous().t(), "unaligned": flat[1:].view(rows, cols), "pitch": wide[:, 3:3 + cols]}
