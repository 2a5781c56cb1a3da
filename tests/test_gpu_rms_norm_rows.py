"""RMS norm backward where a thread takes several rows: more rows than the 1024
workgroups that share them, at 64, 256 and 1024 threads a row, weights of both
types, against 64 bits on the GPU.

Tolerances (u = 2^-24): dx within 256 u of the magnitudes that are added and
half a bf16 spacing; dweight one rounding per row besides 64 u."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


def _half_ulp(x):
    return torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -126))) - 8)


def _inside(got, want, tol, what):
    assert bool(got.isfinite().all()), what
    worst = ((got.double() - want).abs() / tol).max()
    assert float(worst) <= 1.0, f"{what}: {float(worst)} of the tolerance"


# (rows, columns): four rows a workgroup at 64 threads a row (one, two and four
# chunks a thread), a row a workgroup at 256 and 1024; two rows for some
# workgroups, three and more for others
SHAPES = [(4099, 272), (9000, 1008), (8200, 2032), (1025, 2064), (2500, 4080), (3073, 8192),
          (1030, 8208), (2051, 16384)]


@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward_of_many_rows(gpu, shape, wdtype):
    rows, cols = shape
    g = torch.Generator(device=gpu)
    g.manual_seed(rows + cols)

    def matrix(std):
        return (torch.randn(rows, cols + 16, generator=g, device=gpu) * std).bfloat16()[:, :cols]
    s, dy, dres = matrix(3.0), matrix(0.5), matrix(0.25)
    # rows of very different sizes, so that one taken for another shows
    s *= torch.exp2(torch.arange(rows, device=gpu) % 7 - 3.0).bfloat16()[:, None]
    w = (1 + 0.2 * torch.randn(cols, generator=g, device=gpu)).to(wdtype)
    rstd = fp8.rms_norm_fwd(s, w, eps=EPS).rstd
    say("rms_norm_bwd rows", shape, wdtype)
    for extra in (None, dres):
        dx, dw = fp8.rms_norm_bwd(dy, s, rstd, w, dres=extra)
        s64, dy64, w64 = s.double(), dy.double(), w.double()
        r = (s64.square().mean(1, keepdim=True) + EPS).rsqrt()
        _inside(rstd, r[:, 0], 64 * U * r[:, 0], "rstd")
        h, d = s64 * r, dy64 * w64
        want = r * (d - h * (d * h).mean(1, keepdim=True))
        size = r * (d.abs() + h.abs() * (d * h).abs().mean(1, keepdim=True))
        if extra is not None:
            want, size = want + extra.double(), size + extra.double().abs()
        tol = 256 * U * size
        _inside(dx, want, tol + _half_ulp(want.abs() + tol), "dx")
        assert dw.dtype == wdtype
        want, size = (dy64 * h).sum(0), (dy64 * h).abs().sum(0)
        tol = (64 + rows + 8) * U * size
        _inside(dw, want, tol + (_half_ulp(want.abs() + tol) if wdtype == torch.bfloat16 else 0.0), "dweight")
        again = fp8.rms_norm_bwd(dy, s, rstd, w, dres=extra)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
