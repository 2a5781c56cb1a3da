"""NaN in runs of rows of a column: a scale of the transposed codes is that of
the column's other values, whose codes stay as they are without the NaN, and a
NaN's own code is NaN.  Runs are as long as what one thread holds of a column
(four or eight rows) and longer; the column's largest value is near them."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

NAN = float("nan")
# (first row, rows, column): in the block's first rows, which hold its largest
# values, beside them, a whole block of a column, the ragged last tile
RUNS = [(8, 8, 0), (4, 4, 5), (0, 16, 17), (24, 8, 17), (32, 64, 40), (0, 128, 90), (60, 4, 127), (128, 8, 130), (129, 15, 143)]
ROWS, COLS = 144, 144


def _randn(gpu, seed):
    x = torch.randn(ROWS, COLS, generator=torch.Generator().manual_seed(seed))
    x[:16] *= 100
    x[128:132] *= 100
    return x.bfloat16().to(gpu)


def _mask(gpu):
    m = torch.zeros(ROWS, COLS, dtype=torch.bool)
    for first, n, col in RUNS:
        m[first:first + n, col] = True
    return m.to(gpu)


def _same_but_nan(q, recip, want, want_recip, mask, what):
    assert torch.equal(recip, want_recip), what
    assert torch.equal(q[~mask], want[~mask]), what
    assert ((q[mask] & 0x7F) == 0x7F).all(), what


@pytest.mark.parametrize("weighted", [False, True])
def test_gather(gpu, weighted):
    mask = _mask(gpu)
    x = _randn(gpu, 1)
    clean = torch.where(mask, 0.0, x)
    t = fp8.moe_sort(torch.zeros(ROWS, 1, dtype=torch.int64, device=gpu), 1, align=16)
    assert t.source.shape == (ROWS,)
    w = torch.full((ROWS, 1), 2.0, device=gpu)

    def call(x):
        if weighted:
            return fp8.moe_combine_bwd(x, None, t, w, dy=False, q=True, qt=True, need_dweight=False)[0]
        return fp8.moe_gather(x, t, y=False, q=True, qt=True)
    say("moe_gather, NaN columns", weighted)
    o, want = call(x.masked_fill(mask, NAN)), call(clean)
    _same_but_nan(o.qt, o.recip_t, want.qt, want.recip_t, mask.t(), "qt")
    _same_but_nan(o.q, o.recip, want.q, want.recip, mask, "q")
    if not weighted:
        q, recip = fp8.fp8_blockwise_quant(clean, transpose=True)
        assert torch.equal(want.qt, q) and torch.equal(want.recip_t, recip)


def test_swiglu_forward(gpu):
    mask = _mask(gpu)
    g, u = _randn(gpu, 2) / 50, _randn(gpu, 3)
    say("swiglu_fwd, NaN columns")

    def call(u):
        return fp8.swiglu_fwd(torch.cat([g, u], 1), y=False, q=True, qt=True, save=True)
    o, want = call(u.masked_fill(mask, NAN)), call(u.masked_fill(mask, 0.0))
    _same_but_nan(o.qt, o.recip_t, want.qt, want.recip_t, mask.t(), "qt")
    _same_but_nan(o.q, o.recip, want.q, want.recip, mask, "q")
    _same_but_nan(o.hq[:, COLS:], o.h_recip[:, 2:], want.hq[:, COLS:], want.h_recip[:, 2:], mask, "hq")


@pytest.mark.parametrize("codes", [False, True])
def test_swiglu_backward(gpu, codes):
    mask = _mask(gpu)
    g, u, dy = _randn(gpu, 4) / 50, _randn(gpu, 5), _randn(gpu, 6)
    say("swiglu_bwd, NaN columns", codes)

    def call(u, dy):
        h = torch.cat([g, u], 1)
        if codes:
            f = fp8.swiglu_fwd(h, y=False, save=True)
            return fp8.swiglu_bwd(dy, f.hq, f.h_recip, dh=False, q=True, qt=True, act_qt=True)
        return fp8.swiglu_bwd(dy, h, dh=False, q=True, qt=True, act_qt=True)
    both = torch.cat([mask, mask], 1)
    o, want = call(u, dy.masked_fill(mask, NAN)), call(u, dy.masked_fill(mask, 0.0))
    _same_but_nan(o.qt, o.recip_t, want.qt, want.recip_t, both.t(), "qt of dy's NaN")
    _same_but_nan(o.q, o.recip, want.q, want.recip, both, "q of dy's NaN")
    assert torch.equal(o.act_qt, want.act_qt) and torch.equal(o.act_recip_t, want.act_recip_t)
    o, want = call(u.masked_fill(mask, NAN), dy), call(u.masked_fill(mask, 0.0), dy)
    _same_but_nan(o.act_qt, o.act_recip_t, want.act_qt, want.act_recip_t, mask.t(), "act_qt of u's NaN")
    _same_but_nan(o.qt[:COLS], o.recip_t[:COLS], want.qt[:COLS], want.recip_t[:COLS], mask.t(), "qt of u's NaN")
    assert torch.equal(o.qt[COLS:], want.qt[COLS:])
