"""moe_dispatch and moe_join take the plain tuple that torch.ops.fp8bw.moe_sort
gives (what a traced program has in hand) as they take a MoeTable."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8


@pytest.mark.parametrize("lead", [(10,), (2, 5)])
def test_plain_tuple(lead):
    x = torch.empty(*lead, 64, dtype=torch.bfloat16, device="meta", requires_grad=True)
    w = torch.empty(*lead, 3, device="meta", requires_grad=True)
    table = torch.ops.fp8bw.moe_sort(torch.empty(10, 3, dtype=torch.int32, device="meta"), 4, 128)
    assert not isinstance(table, fp8.MoeTable)
    y = fp8.moe_dispatch(x, table)
    assert fp8.moe_join(y, table).shape == (10, 64)
    fp8.moe_join(y, table, w).sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape
