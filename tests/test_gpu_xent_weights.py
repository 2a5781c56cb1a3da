"""Cross entropy with token weights that are infinite or NaN: they reach dw and
their own token's dh, no other's."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(40, 500, 64), (40, 500, 1600), (300, 33001, 64)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_one_bad_weight(gpu, shape, bad):
    T, V, K = shape
    g = torch.Generator().manual_seed(sum(shape))
    h = torch.randn(T, K, generator=g).bfloat16().to(gpu)
    w = (torch.randn(V, K, generator=g) * 2.0 / K ** 0.5).bfloat16().to(gpu)
    target = torch.randint(0, V, (T,), generator=g).to(gpu)
    dloss = torch.rand(T, generator=g).to(gpu) * 0.5
    dloss[3] = 1.0                             # the largest, so that leaving token 7's out changes no scale
    lse = fp8.linear_xent_fwd(h, w, target)[1]
    dloss[7] = 0.0
    say("xent bad weight", shape, bad)
    want, _ = fp8.linear_xent_bwd(dloss, h, w, target, lse)
    dloss[7] = bad
    dh, dw = fp8.linear_xent_bwd(dloss, h, w, target, lse)
    others = torch.arange(T, device=gpu) != 7
    assert torch.equal(dh[others], want[others])
    assert not bool(dh[7].isfinite().any()) and not bool(dw.isfinite().any())


def test_only_bad_weights(gpu):
    h, w = torch.ones(5, 64, device=gpu).bfloat16(), torch.ones(300, 64, device=gpu).bfloat16()
    target = torch.arange(5, device=gpu)
    target[2] = -100
    lse = fp8.linear_xent_fwd(h, w, target)[1]
    say("xent only bad weights")
    dh, _ = fp8.linear_xent_bwd(torch.full((5,), float("inf"), device=gpu), h, w, target, lse)
    assert not dh[2].any() and bool(dh[[0, 1, 3, 4]].isnan().all())
