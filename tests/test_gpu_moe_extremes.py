"""The experts' operators past 2^31 elements (the last rows come out as they do
alone), and infinities, NaN and subnormals, which stay with their rows."""

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _fill(t, seed):
    g = torch.Generator(device=t.device)
    g.manual_seed(seed)
    for i in range(0, t.shape[0], 1 << 12):
        t[i:i + (1 << 12)].normal_(generator=g)
    return t


def _identity(gpu, tokens, experts=1):
    """The table of one choice each, all of one expert: rows in the tokens' order."""
    expert = torch.zeros(tokens, 1, dtype=torch.int64, device=gpu)
    return fp8.moe_sort(expert, experts, 128)


def test_gather_and_combine_past_32_bits(gpu):
    tokens, cols = 33024, 65536                   # 2.16e9 elements
    x = _fill(torch.empty(tokens, cols, dtype=torch.bfloat16, device=gpu), 1)
    t = _identity(gpu, tokens)
    rows = t.source.shape[0]
    assert rows == tokens
    say("moe_gather long, tiles")
    o = fp8.moe_gather(x, t, y=True, q=True, qt=True)
    tail = slice(tokens - 256, tokens)
    for i in range(0, tokens, 4128):
        assert torch.equal(o.y[i:i + 4128], x[i:i + 4128])
    q, recip = fp8.fp8_blockwise_quant(x[tail])
    qt, recip_t = fp8.fp8_blockwise_quant(x[tail], transpose=True)
    assert torch.equal(o.q[tail], q) and torch.equal(o.recip[tail], recip)
    assert torch.equal(o.qt[:, tail], qt) and torch.equal(o.recip_t[:, -2:], recip_t)
    del o
    say("moe_gather long, rows")
    r = fp8.moe_gather(x, t, y=False, q=True)
    assert torch.equal(r.q[tail], q) and torch.equal(r.recip[tail], recip)
    del r
    w = torch.full((tokens, 1), 0.5, device=gpu)
    say("moe_combine long")
    out = fp8.moe_combine(x, t, w)
    assert torch.equal(out[tail], x[tail] * 0.5)
    say("moe_combine_bwd long")
    d, dw = fp8.moe_combine_bwd(x, out, t, w)
    assert torch.equal(d.y[tail], out[tail])
    want = (x[tail].float() * out[tail].float()).sum(1)
    # positive terms: within 2^-24 (8 * 32 + 10), and torch's own sum within what is left
    assert ((dw[tail, 0] - want).abs() <= 2.0 ** -15 * want).all()


def test_gather_of_wide_strides(gpu):
    tokens, cols, ld = 2200, 256, 1 << 20         # the last token starts at element 2.3e9
    x = _fill(torch.empty(tokens, ld, dtype=torch.bfloat16, device=gpu)[:, -cols:], 2)
    t = _identity(gpu, tokens)
    v = torch.zeros(t.source.shape[0], cols, dtype=torch.bfloat16, device=gpu)
    v[:tokens] = x
    say("moe_gather wide")
    for qt in (False, True):
        o = fp8.moe_gather(x, t, y=True, q=True, qt=qt)
        q, recip = fp8.fp8_blockwise_quant(v)
        assert torch.equal(o.y, v) and torch.equal(o.q, q) and torch.equal(o.recip, recip)
    qt, recip_t = fp8.fp8_blockwise_quant(v, transpose=True)
    assert torch.equal(o.qt, qt) and torch.equal(o.recip_t, recip_t)


def test_swiglu_past_32_bits(gpu):
    rows, ffn = 33024, 65536                      # h: 4.3e9 elements
    h = _fill(torch.empty(rows, 2 * ffn, dtype=torch.bfloat16, device=gpu), 3)
    tail = slice(rows - 256, rows)
    a = fp8.swiglu_fwd(h[tail], q=True, qt=True, save=True)
    for qt in (False, True):
        say("swiglu_fwd long", qt)
        o = fp8.swiglu_fwd(h, q=True, qt=qt, save=True)
        for big, small in ((o.y, a.y), (o.q, a.q), (o.recip, a.recip), (o.hq, a.hq), (o.h_recip, a.h_recip)):
            assert torch.equal(big[tail], small)
    assert torch.equal(o.qt[:, tail], a.qt) and torch.equal(o.recip_t[:, -2:], a.recip_t)
    dy = o.y
    for codes in (False, True):
        args = (o.hq, o.h_recip) if codes else (h, None)
        cut = tuple(None if t is None else t[tail] for t in args)
        small = fp8.swiglu_bwd(dy[tail], cut[0], None if cut[1] is None else cut[1].t().contiguous().t(), q=True, qt=True,
                               act_qt=True)
        say("swiglu_bwd long", codes)
        big = fp8.swiglu_bwd(dy, *args, q=True, qt=True, act_qt=True)
        for b, s in ((big.dh, small.dh), (big.q, small.q), (big.recip, small.recip)):
            assert torch.equal(b[tail], s)
        assert torch.equal(big.qt[:, tail], small.qt) and torch.equal(big.act_qt[:, tail], small.act_qt)
        assert torch.equal(big.recip_t[:, -2:], small.recip_t)
        assert torch.equal(big.act_recip_t[:, -2:], small.act_recip_t)
        del big
        rows_only = fp8.swiglu_bwd(dy, *args, q=True)
        assert torch.equal(rows_only.dh[tail], small.dh) and torch.equal(rows_only.q[tail], small.q)
        del rows_only


def _codes(gpu, rows, cols, seed):
    g = torch.Generator(device=gpu)
    g.manual_seed(seed)
    q = torch.empty(rows, cols, dtype=torch.uint8, device=gpu)
    for i in range(0, rows, 2048):
        q[i:i + 2048].random_(0, 96, generator=g)     # positive codes below 2
    s = torch.rand(cols // 128, rows, device=gpu, generator=g).add_(0.5).t()
    return q, s


def test_grouped_wgrad_past_32_bits(gpu):
    M, N, K = 17408, 384, 131072                  # a: 2.28e9 codes
    a, ra = _codes(gpu, M, K, 4)
    b, rb = _codes(gpu, N, K, 5)
    ends = torch.tensor([K - 1024, K], dtype=torch.int32, device=gpu)
    say("grouped wgrad long operand")
    out = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(a, ra, b, rb, ends)
    tail = slice(M - 512, M)
    cut = torch.tensor([0, 1024], dtype=torch.int32, device=gpu)
    small = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(
        a[tail, K - 1024:].contiguous(), ra[tail, -8:].t().contiguous().t(), b[:, K - 1024:].contiguous(),
        rb[:, -8:].t().contiguous().t(), cut)
    # positive terms: the fp32 sums (matrix instructions within 2^-16, 8 additions)
    # agree within 2^-13, and two roundings to bf16 (2^-8 each) part by 2^-7
    torch.testing.assert_close(out[1, tail].float(), small[1].float(), rtol=2.0 ** -7 + 2.0 ** -13, atol=0)
    del a, b, out, small
    M = N = 16384                                 # 9 groups: 2.4e9 outputs
    a, ra = _codes(gpu, M, 1152, 6)
    b, rb = _codes(gpu, N, 1152, 7)
    ends = torch.arange(128, 1280, 128, dtype=torch.int32, device=gpu)
    say("grouped wgrad long output")
    out = fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(a, ra, b, rb, ends)
    last = fp8.fp8_scaled_gemm_blockwise(a[:, 1024:].contiguous(), ra[:, 8:].t().contiguous().t(),
                                         b[:, 1024:].contiguous(), rb[:, 8:].t().contiguous().t(), b_block="1x128")
    torch.testing.assert_close(out[8].float(), last.float(), rtol=2.0 ** -7 + 2.0 ** -13, atol=0)


def test_grouped_quantizer_past_32_bits(gpu):
    w = _fill(torch.empty(9, 16384 * 16384, dtype=torch.bfloat16, device=gpu), 8).view(9, 16384, 16384)
    for transpose in (False, True):
        say("grouped quantizer long", transpose)
        q, recip = fp8.fp8_blockwise_quant_grouped(w, transpose)
        q8, recip8 = fp8.fp8_blockwise_quant(w[8], "128x128", transpose)
        assert torch.equal(q[8], q8) and torch.equal(recip[8], recip8)


def test_swiglu_of_infinities_and_nan(gpu):
    inf, nan = float("inf"), float("nan")
    h = torch.zeros(16, 512, dtype=torch.bfloat16, device=gpu).normal_()
    plain = fp8.swiglu_fwd(h, q=True, qt=True, save=True)
    dirty = h.clone()
    dirty[3, :6] = torch.tensor([inf, -inf, nan, 1.0, 2.0, -1e38], dtype=torch.bfloat16)
    dirty[3, 256:262] = torch.tensor([1.0, 1.0, 1.0, nan, -inf, 1.0], dtype=torch.bfloat16)
    for qt in (False, True):
        o = fp8.swiglu_fwd(dirty, q=True, qt=qt, save=True)
        g, u = dirty[3, :256].float(), dirty[3, 256:].float()
        want = g / (1 + torch.exp(-g)) * u
        assert torch.equal(o.y[3].isnan(), want.isnan())
        assert torch.equal(o.y[3][want.isinf()].float(), want[want.isinf()])
        clean = [r for r in range(16) if r != 3]
        for big, small in ((o.y, plain.y), (o.q, plain.q), (o.recip, plain.recip), (o.hq, plain.hq),
                           (o.h_recip, plain.h_recip)):
            assert torch.equal(big[clean], small[clean])
    dy = torch.ones(16, 256, dtype=torch.bfloat16, device=gpu)
    a, b = fp8.swiglu_bwd(dy, h, q=True, qt=True), fp8.swiglu_bwd(dy, dirty, q=True, qt=True)
    for x, y in ((a.dh, b.dh), (a.q, b.q), (a.recip, b.recip)):
        assert torch.equal(x[clean], y[clean])


def test_subnormals_are_copied(gpu):
    x = torch.arange(-64, 64, dtype=torch.int16, device=gpu).view(1, 128).repeat(16, 1).view(torch.bfloat16)
    x = torch.where(x.isnan(), torch.zeros_like(x), x)
    t = _identity(gpu, 16)
    for qt in (False, True):
        y = fp8.moe_gather(x, t, qt=qt).y
        assert torch.equal(y[:16].view(torch.int16), x.view(torch.int16))


def test_a_tokens_nan_stays_with_it(gpu):
    torch.manual_seed(9)
    m = fp8.Float8BlockwiseMoE(256, 128, 4, device=gpu)
    x = torch.randn(37, 256, device=gpu, dtype=torch.bfloat16)
    expert = torch.randint(0, 4, (37, 2), device=gpu)
    weight = torch.rand(37, 2, device=gpu)
    bad = x.clone()
    bad[5, 7], bad[11, 9] = float("nan"), float("inf")
    clean = [i for i in range(37) if i not in (5, 11)]
    with torch.no_grad():
        a, b = m(x, expert, weight), m(bad, expert, weight)
    assert torch.equal(a[clean], b[clean]) and not b[5].isfinite().any() and not b[11].isfinite().any()
    x.requires_grad_(), bad.requires_grad_()
    for t in (x, bad):
        m(t, expert, weight).backward(torch.ones_like(x))
    assert torch.equal(x.grad[clean], bad.grad[clean])


# enough slots that every workgroup takes several parts of its run
@pytest.mark.parametrize("tokens, topk, experts, align, wide", [
    ((1 << 22) + 5, 8, 1000, 128, True), ((1 << 23) + 1, 4, 3, 1, False), ((1 << 24) - 1, 1, 40, 128, True),
    (300001, 2, 600, 48, False)])
def test_sort_of_many_slots(gpu, tokens, topk, experts, align, wide):
    g = torch.Generator(device=gpu)
    g.manual_seed(tokens)
    dtype = torch.int64 if wide else torch.int32
    e = torch.randint(-1, experts + 1, (tokens, topk), device=gpu, generator=g, dtype=dtype)   # some are none
    say("moe_sort", tokens, topk, experts, align)
    t = fp8.moe_sort(e, experts, align)
    flat = e.flatten().long()
    has = (flat >= 0) & (flat < experts)
    n = torch.bincount(flat[has], minlength=experts)
    padded = (n + align - 1) // align * align
    end = padded.cumsum(0)
    assert torch.equal(t.group_end.long(), end)
    order = torch.sort(torch.where(has, flat, experts), stable=True).indices[:int(n.sum())]
    chosen = flat[order]
    place = torch.arange(order.numel(), device=gpu) - (n.cumsum(0) - n)[chosen] + (end - padded)[chosen]
    row = torch.full_like(flat, -1)
    row[order] = place
    assert torch.equal(t.row.flatten().long(), row)
    source = torch.full((t.source.numel(),), -1, dtype=torch.int64, device=gpu)
    source[place] = order
    assert torch.equal(t.source.long(), source)
