"""Slots sorted by expert, rows gathered and joined, on the GPU against the
64-bit oracle.

Tolerances (u = 2^-24): tables are exact, and so are copied rows and their
codes (the quantizers' recipe on bf16 values).  combine rounds each product and
each addition: at most 2 topk u of the terms' magnitudes, and half a bf16 step.
Weighted copies round once (u) before their bf16 step or code.  dweight: a
thread adds at most ceil(cols / 2048) 8 products in sequence, a wave 6 times,
then 4 waves: (8 ceil(cols / 2048) + 10) u of the products' magnitudes, and its
type's rounding."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import e4m3, metrics, moe, quant, train
from tests.gpu_util import assert_codes_equal, assert_f32_equal, bits, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _f64(t):
    return t.detach().cpu().double().numpy()


def _close(got, want, tol, what):
    bad = np.abs(got - want) > tol
    if bad.any() or not np.isfinite(got).all():
        i = tuple(b[0] for b in np.nonzero(bad | ~np.isfinite(got)))
        raise AssertionError(f"{what}: {int(bad.sum())} off, first {i}: {got[i]!r} for {want[i]!r}")


def _experts(tokens, topk, experts, seed, dropped=0.0, skew=0.0):
    rng = np.random.default_rng(seed)
    e = rng.integers(0, experts, (tokens, topk))
    if skew:
        e = np.where(rng.random(e.shape) < skew, experts // 2, e)
    if dropped:
        e = np.where(rng.random(e.shape) < dropped, rng.choice([-1, experts, -2 ** 31, 2 ** 31 - 1], e.shape), e)
    return e


def _table(gpu, expert, experts, align, wide=True):
    e = torch.from_numpy(expert).to(torch.int64 if wide else torch.int32).to(gpu)
    return fp8.moe_sort(e, experts, align)


def _check_table(t, expert, experts, align):
    rows = moe.rows_bound(*expert.shape, experts, align)
    row, source, end = moe.sort(expert, experts, align, rows)
    assert t.source.shape == (rows,)
    assert np.array_equal(t.group_end.cpu().numpy(), end)
    assert np.array_equal(t.row.cpu().numpy(), row)
    assert np.array_equal(t.source.cpu().numpy(), source)
    return row, source


# one workgroup and several; one expert, as many as fit, numbers at the edge of
# a power of two; the border between the two ways (4096 slots), partial waves
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("tokens, topk, experts, align", [
    (0, 2, 4, 128), (1, 1, 1, 1), (1, 8, 128, 1), (63, 1, 3, 1), (65, 3, 7, 128), (333, 6, 60, 1), (100, 2, 1024, 128),
    (2048, 2, 16, 128), (2049, 2, 16, 128), (4097, 1, 8, 1), (5000, 3, 33, 16), (16640, 2, 16, 128), (3001, 8, 1000, 5),
    (9000, 64, 256, 128), (20000, 1, 1, 128)])
def test_sort(gpu, tokens, topk, experts, align, wide):
    for seed, (dropped, skew) in enumerate([(0.0, 0.0), (0.3, 0.0), (0.0, 0.9), (1.0, 0.0)]):
        expert = _experts(tokens, topk, experts, seed, dropped, skew)
        if not wide:
            expert = np.clip(expert, -2 ** 31, 2 ** 31 - 1)
        say("moe_sort", tokens, topk, experts, align, wide, dropped, skew)
        _check_table(_table(gpu, expert, experts, align, wide), expert, experts, align)


def test_sort_of_int64_numbers_beyond_int32(gpu):
    expert = np.array([[2 ** 32, 0], [1, 2 ** 32 + 1], [-2 ** 40, 2 ** 62]])
    _check_table(_table(gpu, expert, 2, 1), expert, 2, 1)


def _matrix(gpu, rows, cols, seed, pad=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols + pad, generator=g) * std).bfloat16().to(gpu)[:, :cols]


def _check_exact_codes(q, recip, v, what):
    """Codes of bf16-valued v, exactly as the quantizer makes them."""
    want, want_recip = quant.quant_1x128(bits(torch.from_numpy(v.astype(np.float32)).bfloat16()))
    assert_codes_equal(q.cpu().numpy(), want, what)
    assert_f32_equal(recip.cpu().numpy(), want_recip, what + " scales")


SHAPES = [(1, 8, 128, 5120, 1), (1, 1, 1, 16, 1), (3, 2, 4, 144, 128), (40, 3, 5, 1040, 1), (64, 2, 4, 2064, 16),
          (130, 2, 3, 640, 128), (700, 4, 9, 4112, 1), (300, 6, 16, 512, 128), (520, 1, 2, 8208, 1)]


@pytest.mark.parametrize("tokens, topk, experts, cols, align", SHAPES)
@pytest.mark.parametrize("pad, dropped", [(0, 0.0), (48, 0.3)])
def test_gather(gpu, tokens, topk, experts, cols, align, pad, dropped):
    expert = _experts(tokens, topk, experts, 1, dropped)
    t = _table(gpu, expert, experts, align)
    row, source = _check_table(t, expert, experts, align)
    x = _matrix(gpu, tokens, cols, 2, pad)
    v = moe.gather(_f64(x), source, topk)
    rows = len(source)
    for y, q, qt in ((True, False, False), (False, True, False), (True, True, True)):
        qt = qt and rows % 16 == 0
        say("moe_gather", tokens, topk, experts, cols, align, y, q, qt)
        o = fp8.moe_gather(x, t, y=y, q=q, qt=qt)
        torch.cuda.synchronize()
        assert (o.y is None, o.q is None, o.qt is None) == (not y, not q, not qt)
        if y:
            assert np.array_equal(_f64(o.y), v)
        if q:
            _check_exact_codes(o.q, o.recip, v, "q")
        if qt:
            _check_exact_codes(o.qt, o.recip_t, v.T.copy(), "qt")


def _check_near_codes(q, recip, v, what):
    """Codes of values known to u: reciprocals to 4 u, codes to half a spacing."""
    want, want_recip = train.blocks_1x128(v)
    _close(_f64(recip), want_recip, 4 * U * want_recip, what + " scales")
    _, _, spacing = train.e4m3_neighbours(np.minimum(np.abs(want), 448.0))
    _close(e4m3.decode(q.cpu().numpy()), want, spacing / 2 + 8 * U * np.abs(want), what)


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens, topk, experts, cols, align", SHAPES)
def test_combine_and_its_gradients(gpu, tokens, topk, experts, cols, align, wdtype):
    expert = _experts(tokens, topk, experts, 3, 0.25)
    if tokens > 2:
        expert[1] = -1                          # a token without any expert
    t = _table(gpu, expert, experts, align)
    row, source = _check_table(t, expert, experts, align)
    rows = len(source)
    y, dout = _matrix(gpu, rows, cols, 4, 16), _matrix(gpu, tokens, cols, 5, 8, 1e-3)
    y[torch.from_numpy(source < 0).to(gpu)] = float("nan")      # never read
    g = torch.Generator().manual_seed(6)
    w = torch.rand(tokens, topk, generator=g).to(wdtype).to(gpu)
    y64 = np.nan_to_num(_f64(y))
    say("moe_combine", tokens, topk, experts, cols, align, wdtype)
    for weight in (w, None):
        out = fp8.moe_combine(y, t, weight)
        want, size = moe.combine(y64, row, None if weight is None else _f64(weight))
        tol = 2 * topk * U * size
        _close(_f64(out), want, tol + metrics.bf16_ulp(np.abs(want) + tol) / 2, "out")
        if tokens > 2:
            assert not out[1].any()
    want_dw, size = moe.combine_dweight(_f64(dout), y64, row)
    v = moe.gather(_f64(dout), source, topk, _f64(w))
    for dy, q, qt in ((True, False, False), (False, True, False), (True, True, True)):
        qt = qt and rows % 16 == 0
        say("moe_combine_bwd", tokens, topk, experts, cols, align, dy, q, qt)
        o, dw = fp8.moe_combine_bwd(dout, y, t, w, dy=dy, q=q, qt=qt)
        torch.cuda.synchronize()
        assert dw.dtype == wdtype
        tol = (8 * -(-cols // 2048) + 10) * U * size
        if wdtype == torch.bfloat16:
            tol = tol + metrics.bf16_ulp(np.abs(want_dw) + tol) / 2
        _close(_f64(dw), want_dw, tol, "dweight")
        if dy:
            _close(_f64(o.y), v, U * np.abs(v) + metrics.bf16_ulp(np.abs(v) * (1 + U)) / 2, "dy")
        if q:
            _check_near_codes(o.q, o.recip, v, "q")
        if qt:
            _check_near_codes(o.qt, o.recip_t, v.T.copy(), "qt")
    o, dw = fp8.moe_combine_bwd(dout, None, t, w, need_dweight=False)
    assert dw is None
    _close(_f64(o.y), v, U * np.abs(v) + metrics.bf16_ulp(np.abs(v) * (1 + U)) / 2, "dy alone")


def test_a_malformed_table_reads_and_writes_inside(gpu):
    """Rows and slots outside their ranges count as none."""
    tokens, topk, cols = 5, 2, 256
    row = torch.tensor([[0, 99], [-7, 1], [2 ** 31 - 1, 2], [3, -2 ** 31], [16, 15]], dtype=torch.int32, device=gpu)
    source = torch.full((16,), -1, dtype=torch.int32, device=gpu)
    for r, i in ((0, 0), (1, 3), (2, 5), (3, 6), (15, 9)):
        source[r] = i
    source[4], source[5] = 10, 2 ** 31 - 1          # no such slots
    t = fp8.MoeTable(row, source, torch.tensor([16], dtype=torch.int32, device=gpu))
    x, y = _matrix(gpu, tokens, cols, 7), _matrix(gpu, 16, cols, 8)
    good = source.cpu().numpy().copy()
    good[4:6] = -1
    rows = np.where((row.cpu().numpy() >= 0) & (row.cpu().numpy() < 16), row.cpu().numpy(), -1)
    o = fp8.moe_gather(x, t, q=True, qt=True)
    v = moe.gather(_f64(x), good, topk)
    assert np.array_equal(_f64(o.y), v)
    _check_exact_codes(o.qt, o.recip_t, v.T.copy(), "qt")
    o = fp8.moe_gather(x, t)
    assert np.array_equal(_f64(o.y), v)
    want, size = moe.combine(_f64(y), rows)
    _close(_f64(fp8.moe_combine(y, t)), want, 4 * U * size + metrics.bf16_ulp(size) / 2, "out")


def test_infinities_and_nan_stay_with_their_tokens(gpu):
    expert = np.array([[0, 1], [1, 0], [2, -1], [0, 2]])
    t = _table(gpu, expert, 3, 1)
    x = _matrix(gpu, 4, 128, 9)
    x[1, 3], x[1, 4], x[2, 5] = float("inf"), float("nan"), -float("inf")
    row = t.row.cpu().numpy()
    y = fp8.moe_gather(x, t).y
    assert torch.equal(y[row[1, 0]].view(torch.int16), x[1].view(torch.int16))
    for tok in (0, 3):
        assert torch.equal(y[row[tok, 0]], x[tok])
    out = fp8.moe_combine(y, t)
    assert out[0].isfinite().all() and out[3].isfinite().all()
    assert out[1, 3] == float("inf") and out[1, 4].isnan() and out[2, 5] == -float("inf")


def _check_against_quantizer(t, x, o, weight=None):
    """Every layout of a gather equals the quantizers' of the gathered rows."""
    has = t.source >= 0
    slot = t.source.clamp(min=0).long()
    v = torch.where(has[:, None], x[slot // t.row.shape[1]], 0.0)
    if weight is not None:
        return v.float() * weight.reshape(-1)[slot][:, None] * has[:, None]
    q, recip = fp8.fp8_blockwise_quant(v)
    qt, recip_t = fp8.fp8_blockwise_quant(v, transpose=True)
    assert torch.equal(o.q, q) and torch.equal(o.recip, recip)
    assert torch.equal(o.qt, qt) and torch.equal(o.recip_t, recip_t)
    return v


# many row blocks: even, skewed, empty and single-block experts, one expert, more
# experts than a wave has lanes, unaligned ends
@pytest.mark.parametrize("tokens, topk, experts, align, skew", [
    (4500, 2, 16, 128, 0.0), (4500, 2, 7, 128, 0.8), (3000, 3, 65, 128, 0.5), (9000, 2, 1, 128, 0.0),
    (1100, 8, 256, 128, 0.3), (1100, 8, 300, 128, 0.0), (4160, 2, 5, 1, 0.4), (16640, 2, 16, 128, 0.2)])
def test_gather_of_many_row_blocks(gpu, tokens, topk, experts, align, skew):
    expert = _experts(tokens, topk, experts, 20, 0.05, skew)
    t = _table(gpu, expert, experts, align)
    x = _matrix(gpu, tokens, 1168, 21)
    say("moe_gather, many blocks", tokens, topk, experts, align)
    o = fp8.moe_gather(x, t, y=True, q=True, qt=True)
    v = _check_against_quantizer(t, x, o)
    assert torch.equal(o.y, v)
    w = torch.rand(tokens, topk, generator=torch.Generator().manual_seed(22)).to(gpu)
    y = _matrix(gpu, t.source.shape[0], 1168, 23)
    o, dw = fp8.moe_combine_bwd(x, y, t, w, q=True, qt=True)
    assert torch.equal(o.y, _check_against_quantizer(t, x, o, w).bfloat16())
