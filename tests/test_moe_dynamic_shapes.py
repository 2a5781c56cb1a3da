"""The mixture-of-experts operators under torch.compile with a symbolic token
count, on meta tensors: one trace serves every count."""

import pytest
import torch
import torch._dynamo.testing

import blockwise_scaled_fp8_amd as fp8
from oracle import moe

COUNTS = (7, 40, 65, 300, 1000, 4097)


def _inputs(tokens, hidden, topk, grad, mark):
    x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="meta", requires_grad=grad)
    e = torch.empty(tokens, topk, dtype=torch.int64, device="meta")
    w = torch.empty(tokens, topk, device="meta", requires_grad=grad)
    if mark:
        for t in (x, e, w):
            torch._dynamo.mark_dynamic(t, 0)
    return x, e, w


# A count that is not marked is found to change on the second call.
@pytest.mark.parametrize("mark, traces", [(True, 1), (False, 2)])
@pytest.mark.parametrize("grad", [True, False])
def test_layer(grad, mark, traces):
    torch._dynamo.reset()
    m = fp8.Float8BlockwiseMoE(256, 128, 4, device="meta").requires_grad_(grad)
    backend = torch._dynamo.testing.CompileCounterWithBackend("aot_eager")
    compiled = torch.compile(m, backend=backend, fullgraph=True)
    for tokens in COUNTS:
        x, e, w = _inputs(tokens, 256, 2, grad, mark)
        y = compiled(x, e, w)
        assert y.shape == x.shape
        if grad:
            y.sum().backward()
            assert x.grad.shape == x.shape and w.grad.shape == w.shape
            assert m.w13.grad.shape == m.w13.shape and m.w2.grad.shape == m.w2.shape
    assert backend.frame_count == traces


@pytest.mark.parametrize("experts, topk, align", [(4, 2, 128), (100, 8, 1), (3, 1, 16)])
def test_parts(experts, topk, align):
    torch._dynamo.reset()

    def parts(x, e, w):
        table = fp8.MoeTable(*torch.ops.fp8bw.moe_sort(e, experts, align))
        y = fp8.moe_dispatch(x, table)
        return y, table.source, fp8.moe_join(fp8.swiglu(y), table, w)
    backend = torch._dynamo.testing.CompileCounterWithBackend("aot_eager")
    compiled = torch.compile(parts, backend=backend, fullgraph=True)
    for tokens in COUNTS:
        x, e, w = _inputs(tokens, 64, topk, True, True)
        y, source, out = compiled(x, e, w)
        rows = moe.rows_bound(tokens, topk, experts, align)
        assert y.shape == (rows, 64) and source.shape == (rows,) and out.shape == (tokens, 32)
        out.sum().backward()
        assert x.grad.shape == x.shape and w.grad.shape == w.shape
    assert backend.frame_count == 1


def test_rows_of_the_trace_are_the_librarys():
    for tokens in (0, 1, 2, 5, 63, 64, 300):
        for topk in (1, 2, 8):
            for experts in (1, 3, 16, 1000):
                for align in (1, 7, 128):
                    e = torch.empty(tokens, topk, dtype=torch.int32, device="meta")
                    row, source, end = torch.ops.fp8bw.moe_sort(e, experts, align)
                    assert source.shape[0] == fp8.moe_rows(tokens, topk, experts, align)
                    assert row.shape == e.shape and end.shape == (experts,)
