"""Cross entropy on the tile shapes of few tokens over large vocabularies (64 x
256: at most 64 tokens and 512 tiles of 256 columns; 128 rows: 65 to 128
tokens and 128 such tiles) and over several workspace pieces, element by
element against 64 bits on the GPU.

Tolerances (u = 2^-24): a logit is within dz = (K + 8) u sum|h w|, lse and loss
within dz + 2^-18 + 4 u |lse| and twice that; G is off by its logit's and lse's
error (relative to p) and its rounding to bf16 (2^-8 at most), which dh and dw
add through their products with one fp32 rounding per term and half a bf16
spacing at the end."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IGNORE = -100


def _case(T, V, K, seed, gpu):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, K, generator=g).bfloat16()
    w = (torch.randn(V, K, generator=g) * 2.0 / K ** 0.5).bfloat16()
    target = torch.randint(0, V, (T,), generator=g)
    target[0] = V - 1
    target[torch.arange(T) % 7 == 5] = IGNORE
    return [t.to(gpu) for t in (h, w, target, torch.randn(T, generator=g))]


def _half_ulp(x):
    return torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -126))) - 8)


def _inside(got, want, tol, what):
    worst = ((got.double() - want).abs() / tol).max()
    assert float(worst) <= 1.0, f"{what}: {float(worst)} of the tolerance"


def _check(h, w, target, dloss, loss, lse, dh, dw):
    T, K = h.shape
    V = w.shape[0]
    hf, wf, dl = h.double(), w.double(), dloss.double()
    valid = target != IGNORE
    at = target.clamp(min=0)[:, None]
    want_dw, dw_tol = torch.zeros_like(wf), torch.zeros_like(wf)
    for t0 in range(0, T, 2048):
        r = slice(t0, t0 + 2048)
        z = hf[r] @ wf.t()
        want_lse = torch.logsumexp(z, 1)
        dz = (K + 8) * U * (hf[r].abs() @ wf.abs().t())
        tol = dz.amax(1) + 2.0 ** -18 + 4 * U * want_lse.abs()
        _inside(lse[r], want_lse, tol, "lse")
        want_loss = torch.where(valid[r], want_lse - z.gather(1, at[r])[:, 0], 0.0)
        _inside(loss[r], want_loss, 2 * tol, "loss")
        p = z.sub_(want_lse[:, None]).exp_()
        weight = (dl[r] * valid[r])[:, None]
        g_tol = p * weight.abs() * dz.add_(tol[:, None])
        p.scatter_add_(1, at[r], torch.full_like(weight, -1.0)).mul_(weight)
        g, size = p, p.abs()
        g_tol += 2.0 ** -8 * size
        t = g_tol @ wf.abs() + (V + 8) * U * (size @ wf.abs()) + 1e-37
        want = g @ wf
        _inside(dh[r], want, t + _half_ulp(want.abs() + t), "dh")
        want_dw += g.t().contiguous() @ hf[r]
        dw_tol += g_tol.t().contiguous() @ hf[r].abs() + (T + 8) * U * (size.t().contiguous() @ hf[r].abs())
    dw_tol += 1e-37
    _inside(dw, want_dw, dw_tol + _half_ulp(want_dw.abs() + dw_tol), "dw")


# 64 x 256 with whole and ragged last tiles; 128 rows for the logits, and with
# K = 512 for dH's product too; both at a whole number of slabs and past it
SHAPES = [(1, 131073, 64), (33, 130900, 192), (64, 131073, 64), (64, 131072, 128),
          (65, 32769, 64), (100, 33000, 512), (128, 32769, 192), (127, 40001, 576)]


@pytest.mark.parametrize("shape", SHAPES)
def test_few_tokens(gpu, shape):
    args = _case(*shape, sum(shape), gpu)
    h, w, target, dloss = args
    say("xent tiles", shape)
    loss, lse = fp8.linear_xent_fwd(h, w, target)
    dh, dw = fp8.linear_xent_bwd(dloss, h, w, target, lse)
    _check(*args, loss, lse, dh, dw)
    assert torch.equal(fp8.linear_xent_bwd(dloss, h, w, target, lse, need_dw=False)[0], dh)
    assert torch.equal(fp8.linear_xent_bwd(dloss, h, w, target, lse, need_dh=False)[1], dw)


# five and three pieces, the last one shorter than the others
@pytest.mark.parametrize("shape", [(8192, 40000, 64), (8191, 20481, 128), (4100, 66049, 64)])
def test_several_pieces(gpu, shape):
    args = _case(*shape, sum(shape), gpu)
    h, w, target, dloss = args
    say("xent pieces", shape)
    loss, lse = fp8.linear_xent_fwd(h, w, target)
    dh, dw = fp8.linear_xent_bwd(dloss, h, w, target, lse)
    _check(*args, loss, lse, dh, dw)
