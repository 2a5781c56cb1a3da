"""A compiled mixture-of-experts layer on the GPU: one trace over many token
counts, with the eager layer's bits."""

import pytest
import torch
import torch._dynamo.testing

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _pass(m, fn, x, e, w, dout):
    x, w = x.clone().requires_grad_(), w.clone().requires_grad_()
    m.zero_grad()
    out = fn(x, e, w)
    out.backward(dout)
    return [out.detach(), x.grad, w.grad, m.w13.grad.clone(), m.w2.grad.clone()]


def test_layer_of_symbolic_token_counts(gpu):
    torch._dynamo.reset()
    torch.manual_seed(1)
    m = fp8.Float8BlockwiseMoE(256, 128, 5, device=gpu)
    backend = torch._dynamo.testing.CompileCounterWithBackend("aot_eager")
    compiled = torch.compile(m, backend=backend, fullgraph=True, dynamic=True)
    for tokens in (40, 7, 333, 1024):
        g = torch.Generator().manual_seed(tokens)
        x = torch.randn(tokens, 256, generator=g).bfloat16().to(gpu)
        dout = torch.randn(tokens, 256, generator=g).bfloat16().to(gpu)
        e = torch.randint(-1, 5, (tokens, 2), generator=g).to(gpu)
        w = torch.rand(tokens, 2, generator=g).to(gpu)
        say("compiled MoE", tokens)
        for a, b in zip(_pass(m, compiled, x, e, w, dout), _pass(m, m, x, e, w, dout)):
            assert torch.equal(a, b)
    assert backend.frame_count == 1
