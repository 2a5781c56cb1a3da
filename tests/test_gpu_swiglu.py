"""The gated activation, its 8-bit checkpoint and its backward on the GPU
against the 64-bit oracle.

Tolerances (u = 2^-24): exp2 and the reciprocal are within 1 ulp (2 u) and the
exponent g log2(e) is rounded once, which moves exp by |g| u, so sigmoid is
within (|g| + 6) u; the products behind it add at most 6 u: REL(g) = (|g| + 12) u
of the terms' magnitudes.  1 - s is off by u of 1 where s is near 1, that is
|g| u of the slope's second term: covered by the same (|g| + 12) u of s + |g| s.
bf16 outputs add half their spacing, codes half a spacing of E4M3."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import e4m3, metrics, moe, quant, train
from tests.gpu_util import assert_codes_equal, assert_f32_equal, bits, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24

SHAPES = [(1, 16), (1, 8192), (3, 128), (16, 144), (5, 1040), (48, 528), (130, 640), (144, 2064), (700, 512),
          (2064, 272)]


def _f64(t):
    return t.detach().cpu().double().numpy()


def _matrix(gpu, rows, cols, seed, pad=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols + pad, generator=g) * std).bfloat16().to(gpu)[:, :cols]


def _close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(b[0] for b in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} off, first {i}: {got[i]!r} for {want[i]!r}")


def _check_bf16(got, want, tol, what):
    _close(_f64(got), want, tol + metrics.bf16_ulp(np.abs(want) + tol) / 2, what)


def _check_codes(q, recip, v, tol, what):
    """Codes of values known to tol, blocks of 128 along the columns."""
    want, want_recip = train.blocks_1x128(v)
    got_recip = _f64(recip)
    codes = e4m3.decode(q.cpu().numpy()).astype(np.float64)
    for b in range(want_recip.shape[1]):
        c = slice(128 * b, 128 * b + 128)
        off = tol[:, c].max(axis=1) / 448.0
        _close(got_recip[:, b], want_recip[:, b], off + 4 * U * want_recip[:, b], what + " scales")
        # in units of the block's scale, which is off by off / recip
        rel = (off / want_recip[:, b])[:, None] + 8 * U
        _, _, spacing = train.e4m3_neighbours(np.minimum(np.abs(want[:, c]) * (1 + rel), 448.0))
        _close(codes[:, c], want[:, c], spacing / 2 + rel * np.abs(want[:, c]) + tol[:, c] / want_recip[:, b][:, None],
               what)


def _halves(check, q, recip, v, tol, what):
    ffn, blocks = v.shape[1] // 2, recip.shape[1] // 2
    for h in range(2):
        c, b = slice(h * ffn, (h + 1) * ffn), slice(h * blocks, (h + 1) * blocks)
        check(q[:, c], recip[:, b], v[:, c], tol[:, c], f"{what} half {h}")


@pytest.mark.parametrize("rows, ffn", SHAPES)
@pytest.mark.parametrize("pad", [0, 48])
def test_forward(gpu, rows, ffn, pad):
    h = _matrix(gpu, rows, 2 * ffn, rows + ffn, pad, 2.0)
    h64 = _f64(h)
    v = moe.swiglu(h64)
    tol = (np.abs(h64[:, :ffn]) + 12) * U * np.abs(v)
    for y, q, qt, save in ((True, False, False, False), (False, True, False, True), (True, True, True, True)):
        qt = qt and rows % 16 == 0
        say("swiglu_fwd", rows, ffn, pad, y, q, qt, save)
        o = fp8.swiglu_fwd(h, y=y, q=q, qt=qt, save=save)
        torch.cuda.synchronize()
        if y:
            _check_bf16(o.y, v, tol, "y")
        if q:
            _check_codes(o.q, o.recip, v, tol, "q")
        if qt:
            _check_codes(o.qt, o.recip_t, v.T.copy(), tol.T.copy(), "qt")
        if save:
            hb = bits(h.contiguous())
            for half in range(2):
                c = slice(half * ffn, (half + 1) * ffn)
                want, want_recip = quant.quant_1x128(np.ascontiguousarray(hb[:, c]))
                nb = want_recip.shape[1]
                assert_codes_equal(o.hq.cpu().numpy()[:, c], want, "hq")
                assert_f32_equal(o.h_recip.cpu().numpy()[:, half * nb:(half + 1) * nb], want_recip, "h_recip")


@pytest.mark.parametrize("rows, ffn", SHAPES)
@pytest.mark.parametrize("codes", [False, True])
def test_backward(gpu, rows, ffn, codes):
    h, dy = _matrix(gpu, rows, 2 * ffn, rows + ffn, 16, 2.0), _matrix(gpu, rows, ffn, rows, 8, 0.5)
    recip = None
    if codes:
        o = fp8.swiglu_fwd(h, y=False, save=True)
        h, recip = o.hq, o.h_recip
        h64 = moe.halves_values(h.cpu().numpy(), recip.cpu().numpy())
    else:
        h64 = _f64(h)
    grad, size = moe.swiglu_grad(_f64(dy), h64)
    g = np.abs(h64[:, :ffn])
    tol = (np.tile(g, 2) + 12) * U * size
    # 1 - s: u of 1, times |dy u g s|
    tol[:, :ffn] += 2 * U * np.abs(_f64(dy) * h64[:, ffn:]) * g * moe.sigmoid(h64[:, :ffn])
    if codes:
        tol += 4 * U * size * (1 + np.tile(g, 2))     # the codes' values are products
    v = moe.swiglu(h64)
    for dh, q, t in ((True, False, False), (False, True, False), (True, True, True), (False, False, True)):
        t = t and rows % 16 == 0
        say("swiglu_bwd", rows, ffn, codes, dh, q, t)
        o = fp8.swiglu_bwd(dy, h, recip, dh=dh, q=q, qt=t, act_qt=t)
        torch.cuda.synchronize()
        if dh:
            _check_bf16(o.dh, grad, tol, "dh")
        if q:
            _halves(_check_codes, o.q, o.recip, grad, tol, "q")
        if t:
            _check_codes(o.qt, o.recip_t, grad.T.copy(), tol.T.copy(), "qt")
            tv = (g + 16) * 2 * U * np.abs(v)
            _check_codes(o.act_qt, o.act_recip_t, v.T.copy(), tv.T.copy(), "act_qt")


def test_large_gates(gpu):
    """Gates far on either side: finite values and gradients.

    A sigmoid below 2^-126 is the reciprocal of a number above 2^126, which is
    subnormal, flushed, or 0 where exp(-g) is infinite: it is off by at most
    2^-126 itself, so v by 2^-126 |g u|, dg by 2^-126 |dy u| (1 + |g|) and du by
    2^-126 |dy g|, beside the roundings above (with |g| up to 128 there, where
    exp(-g) is finite)."""
    h = torch.zeros(1, 32, dtype=torch.bfloat16)
    gates = [-3e38, -1e4, -200.0, -104.0, -90.0, -88.0, -20.0, -0.0, 0.0, 20.0, 88.0, 90.0, 200.0, 1e4, 1e30, 1.0]
    h[0, :16] = torch.tensor(gates)
    h[0, 16:] = 2.0
    h = h.to(gpu)
    dy = torch.ones(1, 16, dtype=torch.bfloat16, device=gpu)
    h64 = _f64(h)
    g = np.abs(h64[:, :16])
    lost, rel = 2.0 ** -126, (np.minimum(g, 128) + 12) * U
    v = moe.swiglu(h64)
    with np.errstate(over="ignore"):
        _check_bf16(fp8.swiglu_fwd(h).y, v, rel * np.abs(v) + 2 * g * lost, "y")
    grad, size = moe.swiglu_grad(_f64(dy), h64)
    tol = np.tile(rel, 2) * size
    # 1 - s: u of 1, times |dy u g s|
    tol[:, :16] += 2 * U * 2 * g * moe.sigmoid(h64[:, :16]) + 2 * (1 + g) * lost
    tol[:, 16:] += g * lost
    _check_bf16(fp8.swiglu_bwd(dy, h).dh, grad, tol, "dh")
