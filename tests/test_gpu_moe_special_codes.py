"""What the experts' operators' codes make of NaN and infinities: a NaN becomes the
NaN code and has no part in its block's scale; an infinity makes its block's
reciprocal scale infinite, its own code NaN and the block's other finite codes 0.
Everything else is as without them."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
ROWS, COLS = 272, 400
NANS = [(0, 0), (5, 127), (130, 128), (131, 399), (271, 383)]
INFS = [(17, 3, INF), (140, 250, -INF), (200, 399, INF), (271, 0, -INF)]


def _dirty(clean):
    x = clean.clone()
    for r, c in NANS:
        x[r, c] = NAN
    for r, c, v in INFS:
        x[r, c] = v
    return x


def _zeroed(clean):
    x = clean.clone()
    for r, c in NANS:
        x[r, c] = 0.0
    return x


def _check(q, recip, want, want_recip, what, transposed=False, offset=0, block0=0):
    """q of the dirty values against the codes of the zeroed ones; an infinity's
    block is the 128 columns around it (of the transpose: rows)."""
    q, recip, want, want_recip = (t.clone() for t in (q, recip, want, want_recip))
    blocks = []
    for r, c, _ in INFS:
        i, j = (offset + c, r) if transposed else (r, offset + c)
        first = j - j % 128 if transposed else offset + c - c % 128
        last = min(first + 128, ROWS if transposed else offset + COLS)
        kb = j // 128 if transposed else block0 + c // 128
        blocks.append((i, first, last, kb, j))
    nans = [(offset + c, r) if transposed else (r, offset + c) for r, c in NANS]
    infinite = torch.zeros_like(q, dtype=torch.bool)
    for i, first, last, kb, j in blocks:
        assert recip[i, kb] == INF, what
        recip[i, kb] = want_recip[i, kb]
        infinite[i, first:last] = True
        assert (q[i, j] & 0x7F) == 0x7F, what
        q[i, j] = 0
    for i, j in nans:
        assert (q[i, j] & 0x7F) == 0x7F, what
        q[i, j], want[i, j] = 0, 0
    assert not (q[infinite] & 0x7F).any(), what
    assert torch.equal(q[~infinite], want[~infinite]), what
    assert torch.equal(recip, want_recip), what


def _randn(gpu, rows, cols, seed):
    return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)).bfloat16().to(gpu)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("tiles", [False, True])
def test_gather(gpu, weighted, tiles):
    x = _randn(gpu, ROWS, COLS, 1)
    t = fp8.moe_sort(torch.zeros(ROWS, 1, dtype=torch.int64, device=gpu), 1, align=16)
    w = torch.full((ROWS, 1), 0.5, device=gpu)

    def call(x):
        if weighted:
            return fp8.moe_combine_bwd(x, None, t, w, dy=False, q=True, qt=tiles, need_dweight=False)[0]
        return fp8.moe_gather(x, t, y=False, q=True, qt=tiles)
    say("special codes, gather", weighted, tiles)
    o, want = call(_dirty(x)), call(_zeroed(x))
    _check(o.q, o.recip, want.q, want.recip, "q")
    if tiles:
        _check(o.qt, o.recip_t, want.qt, want.recip_t, "qt", transposed=True)
    if not weighted:          # and those of finite values are the quantizers'
        q, recip = fp8.fp8_blockwise_quant(_zeroed(x))
        assert torch.equal(want.q, q) and torch.equal(want.recip, recip)


@pytest.mark.parametrize("tiles", [False, True])
def test_swiglu_forward(gpu, tiles):
    g, u = _randn(gpu, ROWS, COLS, 2).abs() + 0.25, _randn(gpu, ROWS, COLS, 3)

    def call(u):
        return fp8.swiglu_fwd(torch.cat([g, u], 1), y=False, q=True, qt=tiles, save=True)
    say("special codes, swiglu_fwd", tiles)
    o, want = call(_dirty(u)), call(_zeroed(u))
    _check(o.q, o.recip, want.q, want.recip, "q")
    if tiles:
        _check(o.qt, o.recip_t, want.qt, want.recip_t, "qt", transposed=True)
    half = want.h_recip.shape[1] // 2
    _check(o.hq, o.h_recip, want.hq, want.h_recip, "hq", offset=COLS, block0=half)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("codes", [False, True])
def test_swiglu_backward(gpu, codes, tiles):
    g, u = _randn(gpu, ROWS, COLS, 4).abs() + 0.25, _randn(gpu, ROWS, COLS, 5).abs() + 0.25
    dy = _randn(gpu, ROWS, COLS, 6)
    h, recip = torch.cat([g, u], 1), None
    if codes:
        f = fp8.swiglu_fwd(h, y=False, save=True)
        h, recip = f.hq, f.h_recip

    def call(dy):
        return fp8.swiglu_bwd(dy, h, recip, dh=False, q=True, qt=tiles, act_qt=tiles)
    say("special codes, swiglu_bwd", codes, tiles)
    o, want = call(_dirty(dy)), call(_zeroed(dy))
    half = want.recip.shape[1] // 2
    for k in range(2):
        c, b = slice(k * COLS, (k + 1) * COLS), slice(k * half, (k + 1) * half)
        _check(o.q[:, c], o.recip[:, b], want.q[:, c], want.recip[:, b], "q")
        if tiles:
            _check(o.qt[c], o.recip_t[c], want.qt[c], want.recip_t[c], "qt", transposed=True)
    if tiles:
        assert torch.equal(o.act_qt, want.act_qt) and torch.equal(o.act_recip_t, want.act_recip_t)
