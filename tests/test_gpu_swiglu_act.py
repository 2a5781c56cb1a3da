"""The activation's transposed codes made again without any gradient: the bits of
the call that computes both, from bf16 and from a checkpoint; and the layer with
only its second weights trained, whose backward multiplies nothing else."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from blockwise_scaled_fp8_amd import ops
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _randn(gpu, *shape, seed=0, pad=0):
    t = torch.randn(*shape[:-1], shape[-1] + pad, generator=torch.Generator().manual_seed(seed))
    return t.bfloat16().to(gpu)[..., :shape[-1]]


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("rows, ffn, pad", [(16, 16, 0), (144, 272, 16), (128, 128, 0), (1040, 528, 48)])
def test_codes_alone(gpu, rows, ffn, pad, codes):
    h, dy = _randn(gpu, rows, 2 * ffn, seed=1, pad=pad), _randn(gpu, rows, ffn, seed=2)
    recip = None
    if codes:
        f = fp8.swiglu_fwd(h, y=False, save=True)
        wide = torch.zeros(rows, 2 * ffn + pad, dtype=torch.uint8, device=gpu)
        wide[:, :2 * ffn] = f.hq
        h, recip = wide[:, :2 * ffn], f.h_recip.contiguous() if pad else f.h_recip
    say("swiglu_bwd, act_qt alone", rows, ffn, codes)
    want = fp8.swiglu_bwd(dy, h, recip, dh=False, qt=True, act_qt=True)
    for given in (None, dy):
        o = fp8.swiglu_bwd(given, h, recip, dh=False, act_qt=True)
        assert o.dh is None and o.q is None and o.qt is None
        assert torch.equal(o.act_qt, want.act_qt) and torch.equal(o.act_recip_t, want.act_recip_t)
    if not codes:
        f = fp8.swiglu_fwd(h, y=False, qt=True)
        assert torch.equal(o.act_qt, f.qt) and torch.equal(o.act_recip_t, f.recip_t)


def test_refusals(gpu):
    h = _randn(gpu, 32, 64)
    with pytest.raises(ValueError, match="HIP"):
        fp8.swiglu_bwd(None, h)
    with pytest.raises(ValueError):
        fp8.swiglu_bwd(None, h[:, :63], dh=False, act_qt=True)
    with pytest.raises(ValueError):
        fp8.swiglu_bwd(None, h[0], dh=False, act_qt=True)
    with pytest.raises(ValueError):
        fp8.swiglu_bwd(None, h, torch.ones(32, 2, device=gpu), dh=False, act_qt=True)
    with pytest.raises(fp8.FP8BWError):
        fp8.swiglu_bwd(None, h[:24], dh=False, act_qt=True)          # rows % 16
    for empty in (h[:0], h[:, :0]):
        o = fp8.swiglu_bwd(None, empty, dh=False, act_qt=True)
        assert o.act_qt.shape == (empty.shape[1] // 2, empty.shape[0])


def test_layer_with_second_weights_alone_multiplies_nothing_else(gpu, monkeypatch):
    torch.manual_seed(3)
    m = fp8.Float8BlockwiseMoE(256, 384, 5, device=gpu)
    x, dout = _randn(gpu, 300, 256, seed=4), _randn(gpu, 300, 256, seed=5)
    g = torch.Generator().manual_seed(6)
    e, w = torch.randint(-1, 5, (300, 2), generator=g).to(gpu), torch.rand(300, 2, generator=g).to(gpu)
    m(x, e, w).backward(dout)
    want = m.w2.grad.clone()
    calls = []
    for name in ("fp8_scaled_grouped_gemm_blockwise", "fp8_blockwise_quant_grouped", "moe_combine_bwd", "swiglu_bwd",
                 "fp8_scaled_grouped_gemm_blockwise_wgrad"):
        def spy(*a, name=name, fn=getattr(ops, name), **kw):
            calls.append((name, kw))
            return fn(*a, **kw)
        monkeypatch.setattr(ops, name, spy)
    m.w13.requires_grad_(False)
    m.zero_grad()
    out = m(x, e, w)
    calls.clear()
    say("MoE, dW2 alone")
    out.backward(dout)
    assert torch.equal(m.w2.grad, want)
    assert [c[0] for c in calls] == ["moe_combine_bwd", "swiglu_bwd", "fp8_scaled_grouped_gemm_blockwise_wgrad"]
    assert not calls[0][1]["q"] and calls[0][1]["qt"]
