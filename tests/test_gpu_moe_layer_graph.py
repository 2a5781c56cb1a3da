"""A captured training step of Float8BlockwiseMoE through autograd, replayed with new
tokens, routings and gradients in its inputs and eager work between: the eager step's
bits.  No eager graph of the leaves is alive while the step is captured."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TOKENS, HIDDEN, EXPERTS, TOPK = 400, 256, 6, 2


def _fill(x, e, w, dout, seed):
    g = torch.Generator().manual_seed(seed)
    with torch.no_grad():
        x.copy_(torch.randn(TOKENS, HIDDEN, generator=g))
        dout.copy_(torch.randn(TOKENS, HIDDEN, generator=g))
        e.copy_(torch.randint(-1, EXPERTS, (TOKENS, TOPK), generator=g))
        w.copy_(torch.rand(TOKENS, TOPK, generator=g))


@pytest.mark.parametrize("frozen", [(), ("w13",), ("w2",), ("w13", "w2")])
def test_step(gpu, frozen):
    torch.manual_seed(1)
    m = fp8.Float8BlockwiseMoE(HIDDEN, 384, EXPERTS, device=gpu)
    for name in frozen:
        getattr(m, name).requires_grad_(False)
    x = torch.empty(TOKENS, HIDDEN, dtype=torch.bfloat16, device=gpu, requires_grad=True)
    w = torch.empty(TOKENS, TOPK, device=gpu, requires_grad=True)
    e = torch.empty(TOKENS, TOPK, dtype=torch.int64, device=gpu)
    dout = torch.empty(TOKENS, HIDDEN, dtype=torch.bfloat16, device=gpu)
    leaves = [x, w, *(p for p in m.parameters() if p.requires_grad)]

    def step():
        out = m(x, e, w)
        return [out.detach(), *torch.autograd.grad(out, leaves, dout)]
    _fill(x, e, w, dout, 0)
    say("MoE step graph: eager", frozen)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("MoE step graph: capture")
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (2, 3, 4):
        _fill(x, e, w, dout, seed)
        want = [t.clone() for t in step()]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        say("MoE step graph: replay", seed)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (seed, i)
