"""The mixture-of-experts operators together on the GPU, as a layer uses them:
the module equals the entry points it calls and, within what FP8 operands
allow, the layer's formula in 64 bits; every subset of gradients, odd routings,
graphs, streams, two layers at once."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import moe
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _randn(gpu, *shape, seed=0, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(gpu)


def _route(gpu, tokens, topk, experts, seed=0, dropped=0.1):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(tokens, experts, generator=g) + torch.randn(experts, generator=g)
    top = torch.topk(torch.softmax(logits, 1), topk, dim=1)
    e = top.indices.masked_fill(torch.rand(tokens, topk, generator=g) < dropped, -1)
    return e.to(gpu), (top.values / top.values.sum(1, keepdim=True)).to(gpu)


def _layer(gpu, hidden=256, ffn=384, experts=5, seed=1):
    torch.manual_seed(seed)
    return fp8.Float8BlockwiseMoE(hidden, ffn, experts, device=gpu)


def _by_hand(m, x, e, w, dout):
    """The layer's calls, one by one."""
    t = fp8.moe_sort(e, m.experts, align=128)
    xs = fp8.moe_gather(x, t, y=False, q=True, qt=True)
    gemm, quant = fp8.fp8_scaled_grouped_gemm_blockwise, fp8.fp8_blockwise_quant_grouped
    h = gemm(xs.q, xs.recip, *quant(m.w13.detach()), t.group_end)
    a = fp8.swiglu_fwd(h, y=False, q=True, save=True)
    y = gemm(a.q, a.recip, *quant(m.w2.detach()), t.group_end)
    out = fp8.moe_combine(y, t, w)
    dy, dw = fp8.moe_combine_bwd(dout, y, t, w, dy=False, q=True, qt=True)
    da = gemm(dy.q, dy.recip, *quant(m.w2.detach(), transpose=True), t.group_end)
    g = fp8.swiglu_bwd(da, a.hq, a.h_recip, dh=False, q=True, qt=True, act_qt=True)
    wgrad = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad
    dw2 = wgrad(dy.qt, dy.recip_t, g.act_qt, g.act_recip_t, t.group_end)
    dw13 = wgrad(g.qt, g.recip_t, xs.qt, xs.recip_t, t.group_end)
    dx = fp8.moe_combine(gemm(g.q, g.recip, *quant(m.w13.detach(), transpose=True), t.group_end), t)
    return [out, dx, dw, dw13, dw2]


def _module(m, x, e, w, dout, need=(True,) * 4):
    ts = [x.detach().clone(), w.detach().clone(), m.w13, m.w2]
    for t, n in zip(ts, need):
        t.requires_grad_(n)
        t.grad = None
    out = m(ts[0], e, ts[1])
    if any(need):
        out.backward(dout)
    return [out.detach(), *(t.grad for t in ts)]


@pytest.mark.parametrize("tokens", [1, 70, 333, 1024])
def test_module_is_the_entry_points(gpu, tokens):
    m = _layer(gpu)
    x, dout = _randn(gpu, tokens, 256, seed=2), _randn(gpu, tokens, 256, seed=3)
    e, w = _route(gpu, tokens, 2, 5, seed=4)
    say("MoE module", tokens)
    for a, b in zip(_module(m, x, e, w, dout), _by_hand(m, x, e, w, dout)):
        assert torch.equal(a, b)


def _formula(m, x, e, w, dout):
    """The layer and its gradients in 64 bits, without any quantization."""
    x, w, dout, w13, w2 = (t.detach().cpu().double().numpy() for t in (x, w, dout, m.w13, m.w2))
    e = e.cpu().numpy()
    out, dx, dw = np.zeros_like(x), np.zeros_like(x), np.zeros_like(w)
    dw13, dw2 = np.zeros_like(w13), np.zeros_like(w2)
    for k in range(m.experts):
        tok, slot = np.nonzero(e == k)
        h = x[tok] @ w13[k].T
        a = moe.swiglu(h)
        y = a @ w2[k].T
        np.add.at(out, tok, w[tok, slot][:, None] * y)
        dw[tok, slot] = (dout[tok] * y).sum(1)
        dy = w[tok, slot][:, None] * dout[tok]
        dw2[k] = dy.T @ a
        dh, _ = moe.swiglu_grad(dy @ w2[k], h)
        dw13[k] = dh.T @ x[tok]
        np.add.at(dx, tok, dh @ w13[k])
    return [out, dx, dw, dw13, dw2]


@pytest.mark.parametrize("tokens", [200, 1500])
def test_layer_against_its_formula(gpu, tokens):
    """Each E4M3 operand is off by at most 2^-4 of each value (half a step),
    independently from value to value, so a product's 2-norm by at most 2^-4 for
    each of its two operands; the activation passes an error of its input on at
    most 2.2 times (its two factors, silu' <= 1.1).  Forward: two roundings
    before the activation and two behind it, sqrt(2 (2.2^2 + 1)) 2^-4 = 0.21.
    Backward: beside the forward's on both sides, up to four more and the
    checkpoint's: twice that."""
    m = _layer(gpu, experts=3)
    x, dout = _randn(gpu, tokens, 256, seed=5), _randn(gpu, tokens, 256, seed=6)
    e, w = _route(gpu, tokens, 2, 3, seed=7)
    say("MoE formula", tokens)
    for name, got, want in zip(("out", "dx", "dweight", "dw13", "dw2"), _module(m, x, e, w, dout), _formula(m, x, e, w, dout)):
        off = np.linalg.norm(got.cpu().double().numpy() - want) / np.linalg.norm(want)
        print(name, off)
        assert off < (0.21 if name == "out" else 0.42), (name, off)


@pytest.mark.parametrize("need", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (0, 1, 0, 1), (1, 0, 1, 0), (0, 0, 0, 0)])
def test_any_subset_of_gradients(gpu, need):
    m = _layer(gpu)
    x, dout = _randn(gpu, 300, 256, seed=8), _randn(gpu, 300, 256, seed=9)
    e, w = _route(gpu, 300, 2, 5, seed=10)
    whole = _module(m, x, e, w, dout)
    some = _module(m, x, e, w, dout, [bool(n) for n in need])
    if any(need):
        assert torch.equal(some[0], whole[0])
    for n, a, b in zip(need, some[1:], whole[1:]):
        assert (a is None) if not n else torch.equal(a, b)


def test_odd_routings(gpu):
    """No token, none with an expert, all at one expert, an expert named twice by
    a token; int32 numbers, bf16 weights, layouts that are not contiguous."""
    m = _layer(gpu)
    say("MoE odd routings")
    x = _randn(gpu, 0, 256).requires_grad_()
    e, w = torch.zeros(0, 2, dtype=torch.int64, device=gpu), torch.zeros(0, 2, device=gpu, requires_grad=True)
    m(x, e, w).sum().backward()
    assert x.grad.shape == (0, 256) and not m.w13.grad.any() and not m.w2.grad.any()
    with torch.no_grad():
        assert m(x, e, w).shape == (0, 256)
    x, dout = _randn(gpu, 40, 256, seed=11), _randn(gpu, 40, 256, seed=12)
    w = torch.rand(40, 2, generator=torch.Generator().manual_seed(13)).to(gpu)
    out, *grads = _module(m, x, torch.full((40, 2), 5, device=gpu), w, dout)
    assert not any(t.any() for t in (out, *grads))
    one = torch.full((40, 2), 3, device=gpu)
    for a, b in zip(_module(m, x, one, w, dout), _by_hand(m, x, one, w, dout)):
        assert torch.equal(a, b)
    assert not m.w13.grad[[0, 1, 2, 4]].any() and m.w13.grad[3].any()
    # twice the same expert: the same rows, weights added
    y = m(x, one[:, :1], w.sum(1, keepdim=True))
    z = m(x, one, w)
    assert (y.float() - z.float()).norm() <= 2 ** -7 * z.float().norm()
    # layouts
    e, w = _route(gpu, 40, 2, 5, seed=14)
    want = _module(m, x, e, w, dout)
    wide = torch.zeros(40, 512, dtype=torch.bfloat16, device=gpu)
    wide[:, ::2] = x
    got = _module(m, wide[:, ::2], e.int().t().contiguous().t(), w.t().contiguous().t(), dout)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    x3 = x.clone().requires_grad_()
    m(x3.view(4, 10, 256), e.view(4, 10, 2), w.view(4, 10, 2)).sum().backward()     # an expanded gradient
    ones = _module(m, x, e, w, torch.ones_like(dout))
    assert torch.equal(x3.grad, ones[1])
    half = w.bfloat16()
    for a, b in zip(_module(m, x, e, half, dout), _by_hand(m, x, e, half, dout)):
        assert torch.equal(a, b) and a.dtype == b.dtype


def test_inference_is_close_to_training(gpu):
    """Unpadded rows meet other tiles, whose fp32 sums run in another order: the
    same codes, so outputs within a bf16 step of the terms joined."""
    m = _layer(gpu)
    for tokens in (1, 9, 400):
        x = _randn(gpu, tokens, 256, seed=15)
        e, w = _route(gpu, tokens, 2, 5, seed=16)
        with torch.no_grad():
            a = m(x, e, w).float()
        b = m(x.requires_grad_(), e, w).detach().float()
        assert (a - b).norm() <= 2 ** -7 * b.norm()


def test_parts_have_their_gradients(gpu):
    x, dout = _randn(gpu, 60, 144, seed=17).requires_grad_(), _randn(gpu, 60, 144, seed=18)
    e, w = _route(gpu, 60, 3, 7, seed=19)
    w.requires_grad_()
    t = fp8.moe_sort(e, 7, align=1)
    say("moe_dispatch, moe_join, swiglu")
    y = fp8.moe_dispatch(x.view(6, 10, 144), t)
    y.retain_grad()
    fp8.moe_join(y, t, w).backward(dout)
    o, dw = fp8.moe_combine_bwd(dout, y.detach(), t, w.detach())
    assert torch.equal(y.grad, o.y) and torch.equal(w.grad, dw)
    assert torch.equal(x.grad, fp8.moe_combine(o.y, t))
    y = y.detach().requires_grad_()
    fp8.moe_join(y, t).backward(dout)
    assert torch.equal(y.grad, fp8.moe_gather(dout, t).y)
    w2 = w.detach().clone().requires_grad_()          # frozen rows
    fp8.moe_join(y.detach(), t, w2).backward(dout)
    assert torch.equal(w2.grad, dw)
    h, dy = _randn(gpu, 2, 30, 288, seed=20).requires_grad_(), _randn(gpu, 2, 30, 144, seed=21)
    for checkpoint in (False, True):
        h.grad = None
        s = fp8.swiglu(h, checkpoint)
        s.backward(dy)
        f = fp8.swiglu_fwd(h.detach().view(60, 288), save=True)
        args = (f.hq, f.h_recip) if checkpoint else (h.detach().view(60, 288),)
        assert torch.equal(s.view(60, 144), f.y)
        assert torch.equal(h.grad.view(60, 288), fp8.swiglu_bwd(dy.view(60, 144), *args).dh)


def _work(m, x, e, w, dout):
    return _by_hand(m, x, e, w, dout)


def _inputs(gpu, tokens=5000, seed=22):
    # more slots than one workgroup sorts
    m = _layer(gpu, hidden=256, ffn=256, experts=6, seed=seed)
    e, w = _route(gpu, tokens, 2, 6, seed=seed + 1)
    return m, _randn(gpu, tokens, 256, seed=seed + 2), e, w, _randn(gpu, tokens, 256, seed=seed + 3)


def test_two_graphs_replay_beside_eager_work(gpu):
    """Two captured runs with workspaces of their own, replayed in turn with new
    routings in the captured inputs and eager work between: eager bits."""
    sets = [_inputs(gpu, seed=22), _inputs(gpu, tokens=300, seed=40)]
    say("MoE graphs: eager")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            _work(*s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        say("MoE graphs: capture")
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(_work(*s))
    for rep in range(4):
        for i in (rep % 2, 1 - rep % 2):
            m, x, e, w, dout = sets[i]
            ne, nw = _route(gpu, e.shape[0], 2, 6, seed=100 + rep)
            e.copy_(ne)
            w.copy_(nw)
            want = [t.clone() for t in _work(*sets[i])]
            for o in outs[i]:
                o.zero_()
            torch.cuda.synchronize()
            say("MoE graphs: replay", rep, i)
            graphs[i].replay()
            torch.cuda.synchronize()
            for k, (a, b) in enumerate(zip(outs[i], want)):
                assert torch.equal(a, b), (rep, i, k)


def test_two_streams_at_once(gpu):
    sets = [_inputs(gpu, seed=60), _inputs(gpu, tokens=6000, seed=80)]
    want = [[t.clone() for t in _work(*s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    say("MoE streams")
    got = [None, None]
    for _ in range(3):
        for i, (s, stream) in enumerate(zip(sets, streams)):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                got[i] = _work(*s)
    for stream in streams:
        torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_example_runs_with_experts(gpu):
    spec = importlib.util.spec_from_file_location("train_small_lm", os.path.join(ROOT, "examples", "train_small_lm.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    say("example with experts")
    losses = example.train(steps=3, say=lambda *a: None, experts=4)
    assert len(losses) == 3 and all(np.isfinite(losses))
