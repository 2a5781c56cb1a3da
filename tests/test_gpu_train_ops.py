"""The training step's operators together on the GPU: modules and autograd
equal the entry points they call, everything replays from a HIP graph, runs on
another stream, and the example learns."""

import importlib.util
import os

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _randn(gpu, *shape, seed=0, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(gpu)


def test_norm_module_is_the_entry_points(gpu):
    x, r, dy, ds = (_randn(gpu, 2, 50, 272, seed=i) for i in range(4))
    norm = fp8.RMSNorm(272, device=gpu)
    xr, rr = x.clone().requires_grad_(), r.clone().requires_grad_()
    say("RMSNorm module")
    y, s = norm(xr, rr)
    torch.autograd.backward([y, s], [dy, ds])
    o = fp8.rms_norm_fwd(x.view(100, 272), norm.weight, residual=r.view(100, 272))
    dx, dw = fp8.rms_norm_bwd(dy.view(100, 272), o.s, o.rstd, norm.weight, dres=ds.view(100, 272))
    assert torch.equal(y.view(100, 272), o.y) and torch.equal(s.view(100, 272), o.s)
    assert torch.equal(xr.grad.view(100, 272), dx) and torch.equal(rr.grad, xr.grad)
    assert torch.equal(norm.weight.grad, dw)
    # the sum alone, and y alone
    xr.grad = None
    norm(xr, rr)[1].backward(ds)
    assert torch.equal(xr.grad, ds)
    xr.grad = None
    norm(xr).backward(dy)
    want, _ = fp8.rms_norm_bwd(dy.view(100, 272), x.view(100, 272), fp8.rms_norm_fwd(x.view(100, 272), norm.weight).rstd,
                               norm.weight)
    assert torch.equal(xr.grad.view(100, 272), want)


def test_norm_linear_against_norm_then_linear(gpu):
    """The fused block and RMSNorm -> Float8BlockwiseLinear quantize the same
    activation, from fp32 and from its bf16 rounding (2^-9 relative rms at
    most): outputs differ by less than the FP8 rounding both share."""
    M, K, N = 384, 512, 640
    x, r, dy = _randn(gpu, M, K, seed=1), _randn(gpu, M, K, seed=2, std=3.0), _randn(gpu, M, N, seed=3)
    fused = fp8.RMSNormLinear(K, N, device=gpu)
    norm, lin = fp8.RMSNorm(K, device=gpu), fp8.Float8BlockwiseLinear(K, N, device=gpu)
    with torch.no_grad():
        lin.weight.copy_(fused.linear.weight)
    outs = []
    say("RMSNormLinear")
    for run in (lambda a, b: fused(a, b), lambda a, b: (lambda y, s: (lin(y), s))(*norm(a, b))):
        a, b = x.clone().requires_grad_(), r.clone().requires_grad_()
        y, s = run(a, b)
        torch.autograd.backward([y, s], [dy, torch.ones_like(s)])
        outs.append([y, s, a.grad, b.grad])
    outs[0] += [fused.norm.weight.grad, fused.linear.weight.grad]
    outs[1] += [norm.weight.grad, lin.weight.grad]
    assert torch.equal(outs[0][1], outs[1][1])
    # E4M3 rounds to 2^-4 relative at most, 2.6% rms; one of the two operands changes some codes
    for a, b in zip(*outs):
        a, b = a.detach().double(), b.detach().double()
        assert float((a - b).norm() / b.norm()) < 0.03
    with torch.no_grad():
        y, s = fused(x[:50], r[:50])
    assert torch.equal(y, outs[0][0][:50]) and torch.equal(s, outs[0][1][:50])


def test_linear_cross_entropy_reductions(gpu):
    h, w = _randn(gpu, 3, 40, 128, seed=4), _randn(gpu, 999, 128, seed=5, std=0.2)
    t = torch.randint(0, 999, (3, 40), device=gpu)
    t[1] = -100
    say("linear_cross_entropy")
    for reduction in ("mean", "sum", "none"):
        grads, values = [], []
        for kind in ("kernel", "torch"):
            a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
            if kind == "kernel":
                loss = fp8.linear_cross_entropy(a, b, t, reduction=reduction)
            else:
                z = a.float().view(120, 128) @ b.float().t()
                loss = torch.nn.functional.cross_entropy(z, t.view(-1), reduction=reduction)
            loss.sum().backward()
            values.append(loss.detach().reshape(-1))
            grads.append((a.grad.double(), b.grad.double()))
        assert torch.allclose(values[0], values[1], rtol=1e-5, atol=1e-5)
        for x, y in zip(*grads):     # G and the result rounded to bf16, 2^-8 each at most
            assert float((x - y).norm() / y.norm()) < 2.0 ** -7


def _params(gpu):
    return [torch.nn.Parameter(_randn(gpu, *s, seed=10 + i)) for i, s in enumerate(((64, 100), (300,), (7,)))]


@pytest.mark.parametrize("bits", [8, 32])
def test_optimizer_resumes_from_its_state(gpu, bits):
    """Ten steps equal five, a checkpoint, and five more."""
    grads = [[_randn(gpu, *p.shape, seed=100 + 10 * s + i) for i, p in enumerate(_params(gpu))] for s in range(10)]

    def run(params, opt, steps):
        for s in steps:
            for p, g in zip(params, grads[s]):
                p.grad = g
            opt.step()
    make = lambda ps: fp8.AdamW(ps, lr=1e-2, state_bits=bits, master_weights=bits == 32)  # noqa: E731
    say("AdamW optimizer", bits)
    a, b = _params(gpu), _params(gpu)
    oa, ob = make(a), make(b)
    run(a, oa, range(10))
    run(b, ob, range(5))
    c = [torch.nn.Parameter(p.detach().clone()) for p in b]
    oc = make(c)
    oc.load_state_dict(ob.state_dict())
    run(c, oc, range(5, 10))
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    start = _params(gpu)
    assert all(not torch.equal(p, q) for p, q in zip(a, start))
    # a parameter without a gradient stays as it is
    a[1].grad, kept = None, a[1].detach().clone()
    oa.step()
    assert torch.equal(a[1], kept)


def _graph_work(x, r, w, hw, t, dl, state):
    o = fp8.rms_norm_fwd(x, w, residual=r, y=True, q=True, qt=True)
    loss, lse = fp8.linear_xent_fwd(o.y, hw, t)
    dh, dhw = fp8.linear_xent_bwd(dl, o.y, hw, t, lse)
    dx, dw = fp8.rms_norm_bwd(dh, o.s, o.rstd, w)
    work = [s.clone() for s in state]
    fp8.adamw_step([work[0]], [dhw], [work[1]], [work[2]], exp_avg_scales=[work[3]], root_scales=[work[4]], step=3,
                   lr=1e-3, seed=9)
    return [o.s, o.rstd, o.y, o.q, o.recip, o.qt, o.recip_t, loss, lse, dh, dhw, dx, dw, *work]


def _graph_inputs(gpu):
    T, K, V = 1040, 256, 33000
    t = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(3)).to(gpu)
    hw = _randn(gpu, V, K, seed=6, std=0.1)
    n = hw.numel()
    state = [hw.clone(), torch.zeros(n, dtype=torch.uint8, device=gpu), torch.zeros(n, dtype=torch.uint8, device=gpu),
             torch.ones(n // 128, device=gpu), torch.ones(n // 128, device=gpu)]
    return (_randn(gpu, T, K, seed=7), _randn(gpu, T, K, seed=8), torch.ones(K, device=gpu), hw, t,
            torch.full((T,), 1.0 / T, device=gpu), state)


def test_graph_replays_match_eager(gpu):
    """Every operator captured once; each of several replays, with eager work
    and synchronizations between, gives the eager bits."""
    args = _graph_inputs(gpu)
    say("train ops: eager")
    eager = [t.clone() for t in _graph_work(*args)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _graph_work(*args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("train ops: capture")
    with torch.cuda.graph(graph):
        outs = _graph_work(*args)
    for rep in range(4):
        for o in outs:
            o.zero_()
        fp8.rms_norm_fwd(args[0], args[2])
        torch.cuda.synchronize()
        say("train ops: replay", rep)
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, e) in enumerate(zip(outs, eager)):
            assert torch.equal(o, e), f"replay {rep}: output {i}"


def test_another_stream(gpu):
    """On a stream that waits for the inputs' one, with work still queued there."""
    args = _graph_inputs(gpu)
    want = [t.clone() for t in _graph_work(*args)]
    x2 = torch.zeros_like(args[0])
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device=gpu)
    for _ in range(8):
        big = big @ big * 1e-3
    x2.copy_(args[0])                       # queued behind the products
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("train ops: another stream")
    with torch.cuda.stream(side):
        got = _graph_work(x2, *args[1:])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bits", [8, 32])
def test_example_learns(gpu, bits):
    """The synthetic rule's cross entropy is 0.1 log(1000) + the rule's own
    0.33, about 1.0; from log(1000) = 6.9 the loss comes below 3 in 150 steps."""
    spec = importlib.util.spec_from_file_location("train_small_lm", os.path.join(ROOT, "examples", "train_small_lm.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    say("example", bits)
    losses = example.train(steps=150, bits=bits, say=lambda *a: None)
    assert losses[0] > 5.0 and sum(losses[-10:]) / 10 < 3.0, (losses[0], losses[-10:])
