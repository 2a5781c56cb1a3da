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


@pytest.mark.parametrize("layout", ["transposed", "unaligned", "pitch"])
def test_inputs_and_gradients_of_any_layout(gpu, layout):
    M, K, N = 128, 256, 384
    x, r, dy, ds = (_randn(gpu, M, k, seed=i) for i, k in enumerate((K, K, K, K)))
    norm, block = fp8.RMSNorm(K, device=gpu), fp8.RMSNormLinear(K, N, device=gpu)
    w, t = _randn(gpu, 700, K, seed=9, std=0.1), torch.arange(M, device=gpu)
    dl = _randn(gpu, M, N, seed=7)
    other = {id(a): _layouts(a)[layout] for a in (x, r, dy, ds, w, dl)}
    results = []
    say("layouts", layout)
    for pick in (lambda a: a, lambda a: other[id(a)]):
        out = []
        for run in ("norm", "block", "head"):
            a, b, c = (pick(v).detach().requires_grad_() for v in (x, r, w))
            if run == "norm":
                y, s = norm(a, b)
                torch.autograd.backward([y, s], [pick(dy), pick(ds)])
                out += [y, s, a.grad, b.grad]
            elif run == "block":
                y, s = block(a, b)
                torch.autograd.backward([y, s], [pick(dl), pick(ds)])
                out += [y, s, a.grad, b.grad]
                with torch.no_grad():
                    out += list(block(a, b))
            else:
                loss = fp8.linear_cross_entropy(a, c, t)
                loss.backward()
                out += [loss, a.grad, c.grad]
        results.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_a_broadcast_residual(gpu):
    """One row for all tokens: its gradient is the sum over them."""
    M, K = 50, 256
    x, row, dy = _randn(gpu, M, K, seed=1), _randn(gpu, 1, K, seed=2), _randn(gpu, M, K, seed=3)
    norm = fp8.RMSNorm(K, device=gpu)
    results = []
    say("broadcast residual")
    for copy in (False, True):
        a, b = x.clone().requires_grad_(), row.clone().requires_grad_()
        wide = b.expand(M, K)
        y, s = norm(a, wide.contiguous() if copy else wide)
        y.backward(dy)
        results.append((y, s, a.grad, b.grad))
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_changes_in_place_are_recorded(gpu):
    """A graph made before the optimizer's step does not run backward through
    the weights after it; nor one whose input became the norm's sum."""
    p = torch.nn.Parameter(torch.ones(256, device=gpu))
    opt = fp8.AdamW([p], lr=0.1)
    a = torch.ones(256, device=gpu).requires_grad_()
    product = (p * a).sum()
    p.grad = torch.ones_like(p)
    say("version counters")
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        product.backward()
    x = _randn(gpu, 32, 256, seed=1)
    b = torch.ones(256, device=gpu, dtype=torch.bfloat16).requires_grad_()
    product = (x * b).sum()
    fp8.rms_norm_fwd(x, torch.ones(256, device=gpu), residual=x.clone(), s=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        product.backward()
    # tensors without a counter are taken all the same
    with torch.inference_mode():
        q = [torch.ones(256, device=gpu) for _ in range(4)]
        fp8.adamw_step([q[0]], [q[1]], [q[2]], [q[3]], step=1, lr=0.1)
        x = _randn(gpu, 32, 256, seed=1)
        fp8.rms_norm_fwd(x, torch.ones(256, device=gpu), residual=x.clone(), s=x)
    assert bool((q[0] < 1).all())


def test_a_refused_step_changes_nothing(gpu):
    """A wrong gradient scale is refused before any state moves on."""
    p = torch.nn.Parameter(torch.ones(256, device=gpu))
    opt = fp8.AdamW([p], lr=0.1)
    p.grad = torch.ones_like(p)
    opt.step()
    before = p.detach().clone()
    say("refused step")
    with pytest.raises(ValueError):
        opt.step(grad_scale=torch.ones(2, device=gpu))
    assert torch.equal(p, before) and opt.state[p]["step"] == 1


def test_checkpoints_of_other_settings(gpu):
    """States of another width are refused; masters that a checkpoint does not
    have are made from the parameters."""
    def params():
        return [torch.nn.Parameter(_randn(gpu, 300, seed=4))]

    def stepped(**kw):
        ps = params()
        opt = fp8.AdamW(ps, lr=1e-2, **kw)
        ps[0].grad = _randn(gpu, 300, seed=5)
        opt.step()
        return opt.state_dict(), ps
    say("checkpoints")
    for a, b in ((8, 32), (32, 8)):
        with pytest.raises(ValueError, match="state_bits"):
            fp8.AdamW(params(), state_bits=b).load_state_dict(stepped(state_bits=a)[0])
    saved, ps = stepped(state_bits=32)
    opt = fp8.AdamW(ps, lr=1e-2, master_weights=True)
    opt.load_state_dict(saved)
    assert torch.equal(opt.state[ps[0]]["master"], ps[0].detach().float())
    ps[0].grad = _randn(gpu, 300, seed=6)
    opt.step()
    assert torch.equal(opt.state[ps[0]]["master"].bfloat16(), ps[0].detach())


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_loss_in_a_graph(gpu, reduction):
    """The reduced loss of many tokens and its gradients, captured: every
    replay, with eager work in between, gives the eager values."""
    T, V, K = 70000, 300, 64
    h, w = _randn(gpu, T, K, seed=1).requires_grad_(), _randn(gpu, V, K, seed=2, std=0.2).requires_grad_()
    target = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(3)).to(gpu)
    target[::9] = -100

    def work():
        loss = fp8.linear_cross_entropy(h, w, target, reduction=reduction)
        return (loss, *torch.autograd.grad(loss, (h, w)))
    say("loss graph: eager")
    eager = [t.detach().clone() for t in work()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("loss graph: capture")
    with torch.cuda.graph(graph):
        outs = [t.detach() for t in work()]
    for rep in range(5):
        for o in outs:
            o.zero_()
        work()
        (torch.randn(3000000, device=gpu) * 2).sum()
        torch.cuda.synchronize()
        say("loss graph: replay", rep)
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, e) in enumerate(zip(outs, eager)):
            assert torch.equal(o, e), f"replay {rep}: output {i}"
