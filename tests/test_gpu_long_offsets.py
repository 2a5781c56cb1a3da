"""Operands of more than 2^31 elements: the last rows (elements) come out as
they do alone."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _fill(t, seed):
    g = torch.Generator(device=t.device)
    g.manual_seed(seed)
    for i in range(0, t.shape[0], 1 << 14):
        t[i:i + (1 << 14)].normal_(generator=g)
    return t


def test_norm_past_32_bits(gpu):
    rows, cols, ld = 133000, 2048, 16384          # the last row starts at element 2.18e9
    x = _fill(torch.empty(rows, ld, dtype=torch.bfloat16, device=gpu), 1)[:, -cols:]
    w = torch.ones(cols, device=gpu)
    say("rms_norm long")
    o = fp8.rms_norm_fwd(x, w, y=True, q=True)
    tail = slice(rows - 600, rows)                # enough rows to take the same kernel
    a = fp8.rms_norm_fwd(x[tail], w, y=True, q=True)
    for big, small in ((o.y, a.y), (o.q, a.q), (o.recip, a.recip), (o.rstd, a.rstd)):
        assert torch.equal(big[tail], small)
    dx, _ = fp8.rms_norm_bwd(x, x, o.rstd, w)
    assert torch.equal(dx[tail], fp8.rms_norm_bwd(x[tail], x[tail], a.rstd, w)[0])


def test_head_past_32_bits(gpu):
    T, V, K = 70, 134000, 16384                   # W and dW: 2.2e9 elements
    h = _fill(torch.empty(T, K, dtype=torch.bfloat16, device=gpu), 2)
    w = _fill(torch.empty(V, K, dtype=torch.bfloat16, device=gpu), 3).mul_(0.01)
    target = torch.full((T,), V - 1, device=gpu)
    target[: T // 2] = torch.arange(T // 2, device=gpu)
    dloss = torch.ones(T, device=gpu)
    say("linear_xent long")
    loss, lse = fp8.linear_xent_fwd(h, w, target)
    dh, dw = fp8.linear_xent_bwd(dloss, h, w, target, lse)
    z = torch.cat([h.float() @ w[i:i + 8192].float().t() for i in range(0, V, 8192)], 1).double()
    assert float((lse - torch.logsumexp(z, 1)).abs().max()) < 1e-4
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    p[torch.arange(T, device=gpu), target] -= 1
    for rows in (slice(0, 300), slice(V - 300, V)):
        want = p[:, rows].t().contiguous().float() @ h.float()
        # G and dW rounded to bf16, 2^-8 each at most
        assert float((dw[rows].float() - want).norm() / want.norm()) < 2.0 ** -7
    want = sum(p[:, i:i + 8192].float() @ w[i:i + 8192].float() for i in range(0, V, 8192))
    assert float((dh.float() - want).norm() / want.norm()) < 2.0 ** -7


def test_adamw_past_32_bits(gpu):
    n, tail = (1 << 31) + 128 * 9, 128 * 16
    p = torch.zeros(n, dtype=torch.bfloat16, device=gpu)
    g = torch.zeros(n, dtype=torch.bfloat16, device=gpu)
    m, r = (torch.zeros(n, dtype=torch.uint8, device=gpu) for _ in range(2))
    ms, rs = (torch.ones(n // 128, device=gpu) for _ in range(2))
    g[-tail:] = torch.randn(tail, device=gpu).bfloat16()
    p[-tail:] = torch.randn(tail, device=gpu).bfloat16()
    alone = [t[-k:].clone() for t, k in ((p, tail), (g, tail), (m, tail), (r, tail), (ms, 16), (rs, 16))]
    say("adamw long")
    for a in ((p, g, m, r, ms, rs), alone):
        fp8.adamw_step([a[0]], [a[1]], [a[2]], [a[3]], exp_avg_scales=[a[4]], root_scales=[a[5]], step=1, lr=0.1)
    for big, small in zip((p, g, m, r, ms, rs), alone):
        assert torch.equal(big[-small.numel():], small)
    assert not p[:-tail].any() and not m[:-tail].any()
