"""RMS norm on the GPU against the 64-bit oracle.

Tolerances, from the fp32 arithmetic (u = 2^-24): a row's sum of squares takes
at most 64 roundings in sequence, halved by the root, and v two products more,
so rstd, v and the scales are within REL = 64 u relative.  bf16 outputs add
half their spacing (8 significant bits), codes half a spacing of E4M3.  dx: REL
of the magnitudes that are added up.  dweight: one rounding per row."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import e4m3, metrics, train
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
REL = 64 * U
EPS = 1e-6

# one row; widths on both sides of each kernel's limits (512, 2048, 4096,
# 8192 columns), ragged last blocks, few and many rows
SHAPES = [(1, 16), (1, 8192), (3, 128), (5, 1040), (16, 2064), (2, 16384), (600, 496), (513, 528),
          (512, 2048), (515, 2064), (520, 4112), (512, 8208)]


def _inputs(rows, cols, seed, pad=0, wdtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)

    def matrix(std):
        return (torch.randn(rows, cols + pad, generator=g) * std).bfloat16()
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(wdtype)
    return matrix(1.0), matrix(3.0), w, matrix(0.5), matrix(0.25)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _close(got, want, tol, what):
    bad = np.abs(got - want) > tol
    if bad.any() or not np.isfinite(got).all():
        i = tuple(b[0] for b in np.nonzero(bad | ~np.isfinite(got)))
        raise AssertionError(f"{what}: {int(bad.sum())} off, first {i}: {got[i]!r} for {want[i]!r}, tol {np.broadcast_to(tol, got.shape)[i]!r}")


def _half_bf16(want, tol):
    """Half the bf16 spacing at the largest value within tol of want."""
    return metrics.bf16_ulp(np.abs(want) + tol) / 2


def _check_codes(q, recip, v, what):
    """Codes and reciprocals of v (oracle), blocks along its columns."""
    want, want_recip = train.blocks_1x128(v)
    _close(recip, want_recip, REL * want_recip, what + " recip")
    _, _, spacing = train.e4m3_neighbours(np.minimum(np.abs(want), 448.0))
    _close(e4m3.decode(q), want, spacing / 2 + 2 * REL * np.abs(want), what + " codes")


@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(gpu, shape, wdtype):
    rows, cols = shape
    x, r, w, _, _ = _inputs(rows, cols, rows + cols, pad=16, wdtype=wdtype)
    say("rms_norm_fwd", shape, wdtype)
    xd, rd = x.to(gpu)[:, :cols], r.to(gpu)[:, :cols]
    for residual in (None, rd):
        o = fp8.rms_norm_fwd(xd, w.to(gpu), residual=residual, eps=EPS, y=True, q=True, qt=rows % 16 == 0)
        torch.cuda.synchronize()
        s = _f64(x[:, :cols]) if residual is None else train.residual_sum(_f64(x[:, :cols]), _f64(r[:, :cols]))
        assert np.array_equal(_f64(o.s), s)
        v, rstd = train.rms_norm_fwd(s, _f64(w), EPS)
        _close(_f64(o.rstd), rstd, REL * rstd, "rstd")
        _close(_f64(o.y), v, _half_bf16(v, REL * np.abs(v)) + REL * np.abs(v), "y")
        _check_codes(o.q.cpu().numpy(), _f64(o.recip), v, "q")
        if rows % 16 == 0:
            _check_codes(o.qt.cpu().numpy(), _f64(o.recip_t), v.T.copy(), "qt")
        else:
            assert o.qt is None and o.recip_t is None


@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(gpu, shape, wdtype):
    rows, cols = shape
    _, s, w, dy, dres = _inputs(rows, cols, 7 * rows + cols, pad=48, wdtype=wdtype)
    s, dy, dres = s[:, :cols], dy[:, :cols], dres[:, :cols]
    o = fp8.rms_norm_fwd(s.to(gpu), w.to(gpu), eps=EPS)
    say("rms_norm_bwd", shape, wdtype)
    for extra in (None, dres):
        dx, dw = fp8.rms_norm_bwd(dy.to(gpu), s.to(gpu), o.rstd, w.to(gpu),
                                  dres=None if extra is None else extra.to(gpu))
        torch.cuda.synchronize()
        want_dx, want_dw = train.rms_norm_bwd(_f64(dy), _f64(s), _f64(w), EPS, None if extra is None else _f64(extra))
        rstd = _f64(o.rstd)[:, None]
        h, d = np.abs(_f64(s)) * rstd, np.abs(_f64(dy) * _f64(w))
        size = rstd * (d + h * (d * h).mean(axis=1, keepdims=True))
        if extra is not None:
            size = size + np.abs(_f64(extra))
        _close(_f64(dx), want_dx, _half_bf16(want_dx, 4 * REL * size) + 4 * REL * size, "dx")
        assert dw.dtype == wdtype
        size = (np.abs(_f64(dy)) * h).sum(axis=0)
        tol = (REL + (rows + 8) * U) * size
        out = _half_bf16(want_dw, tol) if wdtype == torch.bfloat16 else 0.0
        _close(_f64(dw), want_dw, out + tol, "dweight")


def test_sum_in_place_and_repeats(gpu):
    """s may be written over the residual (or x); equal calls give equal bits."""
    x, r, w, dy, _ = (t.to(gpu) for t in _inputs(700, 4112, 3))
    a = fp8.rms_norm_fwd(x, w, residual=r, q=True)
    for into in ("x", "r"):
        xs, rs = x.clone(), r.clone()
        say("rms_norm in place", into)
        b = fp8.rms_norm_fwd(xs, w, residual=rs, q=True, s=xs if into == "x" else rs)
        for t, u in ((a.s, b.s), (a.rstd, b.rstd), (a.y, b.y), (a.q, b.q), (a.recip, b.recip)):
            assert torch.equal(t, u)
    first = fp8.rms_norm_bwd(dy, a.s, a.rstd, w)
    for _ in range(3):
        again = fp8.rms_norm_bwd(dy, a.s, a.rstd, w)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_zero_rows_of_data_and_empty_calls(gpu):
    """All-zero rows: rstd = eps^-1/2, zeros out, the quantizers' floor scale.
    No rows: nothing to do."""
    w = torch.ones(256, device=gpu)
    x = torch.zeros(16, 256, dtype=torch.bfloat16, device=gpu)
    o = fp8.rms_norm_fwd(x, w, eps=1e-4, q=True, qt=True)
    assert not o.y.any() and not o.q.any() and not o.qt.any()
    assert torch.allclose(o.rstd, torch.full_like(o.rstd, 100.0), rtol=1e-6)
    assert bool((o.recip == 1.0 / (np.float32(448) / np.float32(1e-12))).all())
    dx, dw = fp8.rms_norm_bwd(torch.ones_like(x), x, o.rstd, w)
    assert torch.allclose(dx.float(), torch.full_like(dx, 100.0).float(), rtol=2.0 ** -8) and not dw.any()
    e = fp8.rms_norm_fwd(x[:0], w, q=True, qt=True)
    assert e.y.shape == (0, 256) and e.qt.shape == (256, 0)
    dx, dw = fp8.rms_norm_bwd(x[:0], x[:0], e.rstd, w)
    assert dx.shape == (0, 256) and not dw.any()


def test_outputs_stay_in_bounds(gpu):
    """Nothing outside the columns of a wider buffer is written."""
    rows, cols = 130, 528
    x, r, w, _, _ = (t.to(gpu) for t in _inputs(rows, cols, 5))
    wide = torch.full((rows + 2, cols + 32), 7.0, dtype=torch.bfloat16, device=gpu)
    say("rms_norm canary")
    fp8.rms_norm_fwd(x, w, residual=r, s=wide[1:-1, 16:-16])
    inner = wide[1:-1, 16:-16].clone()
    wide[1:-1, 16:-16] = 7.0
    assert bool((wide == 7.0).all())
    assert np.array_equal(_f64(inner), train.residual_sum(_f64(x), _f64(r)))
