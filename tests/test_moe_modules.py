"""The mixture-of-experts modules without a GPU: shapes through autograd on meta
tensors, and refusals."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8


def _meta(*shape, dtype=torch.bfloat16, grad=False):
    return torch.empty(*shape, device="meta", dtype=dtype, requires_grad=grad)


@pytest.mark.parametrize("lead", [(), (3,), (0,), (2, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_shapes(lead, dtype):
    m = fp8.Float8BlockwiseMoE(256, 128, 4, device="meta")
    x, e = _meta(*lead, 7, 256, grad=True), _meta(*lead, 7, 2, dtype=torch.int64)
    w = _meta(*lead, 7, 2, dtype=dtype, grad=True)
    y = m(x, e, w)
    assert y.shape == x.shape
    y.sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape and w.grad.dtype == dtype
    assert m.w13.grad.shape == m.w13.shape and m.w2.grad.shape == m.w2.shape
    with torch.no_grad():
        assert m(x, e, w).shape == x.shape


def test_parts_shapes():
    e = _meta(10, 3, dtype=torch.int32)
    table = fp8.MoeTable(*torch.ops.fp8bw.moe_sort(e, 4, 128))
    rows = fp8.moe_rows(10, 3, 4)
    assert [t.shape for t in table] == [(10, 3), (rows,), (4,)] and rows == 512
    x, w = _meta(10, 64, grad=True), _meta(10, 3, dtype=torch.float32, grad=True)
    y = fp8.moe_dispatch(x, table)
    assert y.shape == (rows, 64)
    for weight in (w, None):
        out = fp8.moe_join(y, table, weight)
        assert out.shape == (10, 64)
    fp8.moe_join(y, table, w).sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape
    h = _meta(2, 5, 96, grad=True)
    for checkpoint in (False, True):
        s = fp8.swiglu(h, checkpoint)
        assert s.shape == (2, 5, 48)
        s.sum().backward()
        assert h.grad.shape == h.shape


def test_layer_refusals():
    for bad in ((100, 128, 4), (128, 100, 4), (128, 128, 0), (128, 128, 1025)):
        with pytest.raises(ValueError):
            fp8.Float8BlockwiseMoE(*bad, device="meta")
    m = fp8.Float8BlockwiseMoE(128, 128, 2)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP"):
        m(x, torch.zeros(4, 1, dtype=torch.int64), torch.ones(4, 1))
    for e, w in (((4, 2), (4, 1)), ((3, 1), (3, 1)), ((4,), (4,))):
        with pytest.raises(ValueError, match="topk"):
            m(x, torch.zeros(e, dtype=torch.int64), torch.ones(w))
    bound = 1 / 128 ** 0.5
    assert float(m.w13.detach().abs().max()) <= bound and float(m.w2.detach().abs().max()) <= bound
