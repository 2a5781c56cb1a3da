"""Refusals of the mixture-of-experts entry points, without a GPU: every invalid
argument is rejected on the host before any HIP call, and what the binding
refuses never reaches the library."""

import ctypes

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from blockwise_scaled_fp8_amd import _lib
from oracle import moe

OK, NULL, SHAPE, LAYOUT, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5, 6
P = 0x10000  # a 256-byte aligned fake device address; never dereferenced here
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    return fp8.load_library()


def _check(lib, fn, base, want, kw):
    a = dict(base)
    assert set(kw) <= set(a), kw
    a.update(kw)
    assert getattr(lib, fn)(*a.values()) == want, kw
    assert bool(lib.fp8bw_last_error()) == (want != OK)


def _layouts(**kw):
    a = dict(y=P, ld_y=256, q=None, ld_q=256, recip=None, rs_row=1, rs_kb=64, qt=None, ld_qt=64, recip_t=None,
             rst_row=1, rst_kb=256)
    a.update(kw)
    return ctypes.byref(_lib.Layouts(*a.values()))


# Layouts of a [64, 256] result and what is wrong with them.
BAD_LAYOUTS = [
    (ALIGN, dict(y=P + 8)), (LAYOUT, dict(ld_y=248)), (LAYOUT, dict(ld_y=260)), (LAYOUT, dict(ld_y=BIG)),
    (NULL, dict(q=P)), (ALIGN, dict(q=P + 8, recip=P)), (ALIGN, dict(q=P, recip=P + 2)),
    (LAYOUT, dict(q=P, recip=P, ld_q=264)), (LAYOUT, dict(q=P, recip=P, rs_kb=32)),
    (LAYOUT, dict(q=P, recip=P, rs_row=-1)), (NULL, dict(qt=P)), (LAYOUT, dict(qt=P, recip_t=P, ld_qt=48)),
    (LAYOUT, dict(qt=P, recip_t=P, rst_row=0)), (LAYOUT, dict(qt=P, recip_t=P, ld_qt=BIG - 16))]


def test_rows(lib):
    for tokens, topk, experts, align in ((0, 2, 4, 128), (1, 8, 128, 1), (16640, 2, 16, 128), (3, 2, 100, 7), (5, 1, 1, 65536)):
        assert lib.fp8bw_moe_rows(tokens, topk, experts, align) == moe.rows_bound(tokens, topk, experts, align)
    for bad in ((-1, 1, 1, 1), (1 << 24, 1, 1, 1), (1, 0, 1, 1), (1, 65, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                (1, 1, 1, 65537), (BIG, 1, 1, 1), (1, BIG, 1, 1), (1, 1, BIG, 1), (1, 1, 1, BIG), ((1 << 24) - 1, 64, 4, 1)):
        assert lib.fp8bw_moe_rows(*bad) == 0
    assert lib.fp8bw_moe_sort_ws_bytes(4, 2, 8) == 0 and lib.fp8bw_moe_sort_ws_bytes(16640, 2, 16) > 0
    assert lib.fp8bw_moe_sort_ws_bytes(16640, 2, 1025) == 0 and lib.fp8bw_moe_sort_ws_bytes(BIG, 2, 16) == 0


SORT = dict(expert=P, index_bits=64, tokens=16640, topk=2, experts=16, align=128, rows=35200, row=P, source=P, group_end=P,
            ws=P, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("want, kw", [
    (UNSUP, dict(index_bits=16)), (SHAPE, dict(tokens=-1)), (SHAPE, dict(tokens=1 << 24)), (SHAPE, dict(topk=0)),
    (SHAPE, dict(topk=65)), (SHAPE, dict(experts=0)), (SHAPE, dict(experts=1025)), (SHAPE, dict(align=0)),
    (SHAPE, dict(align=65537)), (SHAPE, dict(rows=35199)), (SHAPE, dict(rows=1 << 27)), (SHAPE, dict(rows=-1)),
    (NULL, dict(expert=None)), (NULL, dict(row=None)), (NULL, dict(source=None)), (NULL, dict(group_end=None)),
    (ALIGN, dict(expert=P + 4)), (ALIGN, dict(expert=P + 2, index_bits=32)), (ALIGN, dict(row=P + 1)),
    (ALIGN, dict(source=P + 2)), (ALIGN, dict(group_end=P + 3)), (WS, dict(ws=None)), (WS, dict(ws_bytes=0)),
    (ALIGN, dict(ws=P + 64)), (SHAPE, dict(tokens=(1 << 24) - 1, topk=64, rows=(1 << 27) - 1))])
def test_sort(lib, want, kw):
    _check(lib, "fp8bw_moe_sort", SORT, want, kw)


TABLE = [(SHAPE, dict(tokens=-1)), (SHAPE, dict(tokens=1 << 24)), (SHAPE, dict(topk=0)), (SHAPE, dict(topk=65)),
         (SHAPE, dict(rows=-16)), (SHAPE, dict(rows=1 << 27)), (SHAPE, dict(cols=250)), (SHAPE, dict(cols=65552)),
         (SHAPE, dict(cols=-16)), (SHAPE, dict(rows=0)), (SHAPE, dict(tokens=0)), (SHAPE, dict(rows=(1 << 27) - 16, cols=65536)),
         (NULL, dict(row=None)), (ALIGN, dict(row=P + 2))]

GATHER = dict(x=P, ld_x=256, tokens=20, topk=2, row=P, source=P, rows=64, cols=256, out=_layouts(), stream=None)


@pytest.mark.parametrize("want, kw", TABLE + [
    (NULL, dict(x=None)), (ALIGN, dict(x=P + 8)), (LAYOUT, dict(ld_x=252)), (LAYOUT, dict(ld_x=-256)),
    (NULL, dict(source=None)), (ALIGN, dict(source=P + 2)), (NULL, dict(out=None)),
    (SHAPE, dict(rows=60, out=_layouts(qt=P, recip_t=P))),
    (OK, dict(tokens=0, rows=0, x=None, row=None, source=None, out=None)), (OK, dict(cols=0, x=None, out=None))]
    + [(w, dict(out=_layouts(**k))) for w, k in BAD_LAYOUTS])
def test_gather(lib, want, kw):
    _check(lib, "fp8bw_moe_gather", GATHER, want, kw)


COMBINE = dict(y=P, ld_y=256, weight=P, weight_dtype=1, tokens=20, topk=2, row=P, rows=64, cols=256, out=P, ld_out=256,
               stream=None)


@pytest.mark.parametrize("want, kw", TABLE + [
    (NULL, dict(y=None)), (LAYOUT, dict(ld_y=8)), (NULL, dict(out=None)), (ALIGN, dict(out=P + 4)),
    (LAYOUT, dict(ld_out=255)), (UNSUP, dict(weight_dtype=2)), (ALIGN, dict(weight=P + 2)),
    (ALIGN, dict(weight=P + 1, weight_dtype=0)), (OK, dict(tokens=0, rows=0, y=None, out=None)),
    (OK, dict(cols=0, y=None, out=None))])
def test_combine(lib, want, kw):
    _check(lib, "fp8bw_moe_combine", COMBINE, want, kw)


COMBINE_BWD = dict(dout=P, ld_dout=256, y=P, ld_y=256, weight=P, weight_dtype=1, tokens=20, topk=2, row=P, source=P, rows=64,
                   cols=256, dy=_layouts(), dweight=P, stream=None)


@pytest.mark.parametrize("want, kw", TABLE + [
    (NULL, dict(dout=None)), (LAYOUT, dict(ld_dout=8)), (NULL, dict(y=None)), (LAYOUT, dict(ld_y=8)),
    (ALIGN, dict(y=P + 2)), (NULL, dict(source=None)), (NULL, dict(dy=None)), (UNSUP, dict(weight_dtype=-1)),
    (ALIGN, dict(weight=P + 2)), (ALIGN, dict(dweight=P + 2)), (SHAPE, dict(cols=0)),
    (OK, dict(tokens=0, rows=0, dout=None, dy=None)), (OK, dict(cols=0, dweight=None, dout=None))]
    + [(w, dict(dy=_layouts(**k))) for w, k in BAD_LAYOUTS])
def test_combine_bwd(lib, want, kw):
    _check(lib, "fp8bw_moe_combine_bwd", COMBINE_BWD, want, kw)


SWIGLU_FWD = dict(h=P, ld_h=512, rows=64, ffn=256, out=_layouts(), hq=None, ld_hq=512, h_recip=None, hr_row=1, hr_kb=64,
                  stream=None)
FFN = [(SHAPE, dict(rows=-1)), (SHAPE, dict(rows=1 << 27)), (SHAPE, dict(ffn=250)), (SHAPE, dict(ffn=-16)),
       (SHAPE, dict(ffn=(1 << 20) + 16)), (SHAPE, dict(rows=(1 << 27) - 16, ffn=1 << 20)), (NULL, dict(h=None)),
       (ALIGN, dict(h=P + 8)), (LAYOUT, dict(ld_h=504)), (LAYOUT, dict(ld_h=BIG))]


@pytest.mark.parametrize("want, kw", FFN + [
    (NULL, dict(out=None)), (NULL, dict(hq=P)), (ALIGN, dict(hq=P + 8, h_recip=P)), (LAYOUT, dict(hq=P, h_recip=P, ld_hq=504)),
    (LAYOUT, dict(hq=P, h_recip=P, hr_kb=32)), (SHAPE, dict(rows=60, out=_layouts(qt=P, recip_t=P))),
    (OK, dict(rows=0, h=None, out=None)), (OK, dict(ffn=0, h=None, out=None)), (OK, dict(out=_layouts(y=None)))]
    + [(w, dict(out=_layouts(**k))) for w, k in BAD_LAYOUTS])
def test_swiglu_fwd(lib, want, kw):
    _check(lib, "fp8bw_swiglu_fwd", SWIGLU_FWD, want, kw)


SWIGLU_BWD = dict(dy=P, ld_dy=256, h=P, ld_h=512, h_recip=None, hr_row=1, hr_kb=64, rows=64, ffn=256,
                  dh=_layouts(ld_y=512, ld_q=512, rst_kb=512), act_qt=None, ld_act_qt=64, act_recip_t=None, art_row=1,
                  art_kb=256, stream=None)


@pytest.mark.parametrize("want, kw", FFN + [
    (NULL, dict(dy=None)), (LAYOUT, dict(ld_dy=248)), (NULL, dict(dh=None)), (NULL, dict(h=None, h_recip=P)),
    (LAYOUT, dict(h_recip=P, ld_h=520)), (LAYOUT, dict(h_recip=P, hr_kb=63)), (LAYOUT, dict(dh=_layouts(ld_y=256))),
    (LAYOUT, dict(dh=_layouts(y=None, q=P, recip=P, ld_q=256))),
    (LAYOUT, dict(dh=_layouts(y=None, qt=P, recip_t=P, rst_row=0))), (NULL, dict(act_qt=P)),
    (LAYOUT, dict(act_qt=P, act_recip_t=P, ld_act_qt=48)), (LAYOUT, dict(act_qt=P, act_recip_t=P, art_row=0)),
    (SHAPE, dict(act_qt=P, act_recip_t=P, rows=60)), (OK, dict(rows=0, dy=None, h=None, dh=None)),
    (OK, dict(ffn=0, dy=None, h=None, dh=None)), (OK, dict(dh=_layouts(y=None)))])
def test_swiglu_bwd(lib, want, kw):
    _check(lib, "fp8bw_swiglu_bwd", SWIGLU_BWD, want, kw)


WGRAD = dict(a=P, lda=256, ra=P, ra_s_row=1, ra_s_kb=64, b=P, ldb=256, rb=P, rb_s_row=1, rb_s_kb=96, groups=4, group_end=P,
             M=64, N=96, K=256, out=P, ldo=96, out_s_group=64 * 96, out_dtype=0, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("want, kw", [
    (SHAPE, dict(groups=0)), (SHAPE, dict(groups=(1 << 20) + 1)), (SHAPE, dict(M=-1)), (SHAPE, dict(K=200)),
    (SHAPE, dict(N=(1 << 30) + 1)), (UNSUP, dict(out_dtype=2)), (NULL, dict(a=None)), (NULL, dict(b=None)),
    (NULL, dict(ra=None)), (NULL, dict(rb=None)), (NULL, dict(group_end=None)), (NULL, dict(out=None)),
    (ALIGN, dict(a=P + 8)), (ALIGN, dict(b=P + 1)), (ALIGN, dict(ra=P + 2)), (ALIGN, dict(out=P + 8)),
    (ALIGN, dict(group_end=P + 2)), (LAYOUT, dict(lda=240)), (LAYOUT, dict(ldb=264)), (LAYOUT, dict(ra_s_kb=32)),
    (LAYOUT, dict(rb_s_row=-1)), (LAYOUT, dict(ldo=95)), (LAYOUT, dict(ldo=BIG)), (LAYOUT, dict(out_s_group=64 * 96 - 1)),
    (LAYOUT, dict(out_s_group=BIG)), (LAYOUT, dict(lda=BIG - 16)),
    (UNSUP, dict(M=1 << 20, N=1 << 20, ldo=1 << 20, out_s_group=1 << 40, ra_s_kb=1 << 20, rb_s_kb=1 << 20)),
    (OK, dict(M=0, a=None, out=None)), (OK, dict(N=0, b=None, out=None))])
def test_grouped_wgrad(lib, want, kw):
    _check(lib, "fp8_scaled_grouped_gemm_blockwise_wgrad", WGRAD, want, kw)


QUANT = dict(x=P, rows=256, cols=128, ld_x=128, x_s_group=256 * 128, groups=3, transpose=0, q=P, ld_q=128, q_s_group=256 * 128,
             recip=P, rs_row=1, rs_kb=2, recip_s_group=2, stream=None)


@pytest.mark.parametrize("want, kw", [
    (SHAPE, dict(groups=0)), (SHAPE, dict(groups=65536)), (UNSUP, dict(transpose=2)), (SHAPE, dict(rows=-1)),
    (SHAPE, dict(cols=120)), (SHAPE, dict(rows=250, transpose=1)), (SHAPE, dict(rows=1 << 30, cols=1 << 30)),
    (NULL, dict(x=None)), (NULL, dict(q=None)), (NULL, dict(recip=None)), (ALIGN, dict(x=P + 2)), (ALIGN, dict(q=P + 8)),
    (LAYOUT, dict(ld_x=120)), (LAYOUT, dict(ld_q=136)), (LAYOUT, dict(ld_q=128, transpose=1)), (LAYOUT, dict(rs_row=0)),
    (LAYOUT, dict(x_s_group=-8)), (LAYOUT, dict(x_s_group=12)), (LAYOUT, dict(x_s_group=BIG)),
    (LAYOUT, dict(q_s_group=256 * 128 - 16)), (LAYOUT, dict(q_s_group=256 * 128 + 8)), (LAYOUT, dict(recip_s_group=1)),
    (OK, dict(rows=0, x=None)), (OK, dict(cols=0, q=None))])
def test_grouped_quantizer(lib, want, kw):
    _check(lib, "fp8_blockwise_quant_grouped", QUANT, want, kw)


def test_the_binding_takes_gpu_tensors_only():
    e = torch.zeros(4, 2, dtype=torch.int64)
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    t = fp8.MoeTable(e.int(), torch.zeros(8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    codes, scales = torch.zeros(16, 128, dtype=torch.uint8), torch.ones(16, 1)
    for call in (lambda: fp8.moe_sort(e, 2), lambda: fp8.moe_gather(x, t), lambda: fp8.moe_combine(x, t),
                 lambda: fp8.moe_combine_bwd(x, x, t, torch.ones(4, 2)), lambda: fp8.swiglu_fwd(x),
                 lambda: fp8.swiglu_bwd(x, x), lambda: fp8.fp8_blockwise_quant_grouped(x[None]),
                 lambda: fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(codes, scales, codes, scales, t.group_end)):
        with pytest.raises(ValueError, match="HIP"):
            call()


def test_grouped_wgrad_workspace(lib):
    need = lib.fp8bw_grouped_wgrad_ws_bytes(512, 512, 32768, 1)
    assert need >= 2 * 512 * 512 * 4 and need % 256 == 0
    assert lib.fp8bw_grouped_wgrad_ws_bytes(8192, 5120, 33280, 16) == 0
    for bad in ((512, 512, 32768, 0), (0, 512, 32768, 1), (512, 512, 32760, 1), (-1, 512, 32768, 1), (BIG, 1, 128, 1)):
        assert lib.fp8bw_grouped_wgrad_ws_bytes(*bad) == 0
    long = dict(WGRAD, groups=1, M=512, N=512, K=32768, lda=32768, ldb=32768, ra_s_kb=512, rb_s_kb=512, ldo=512,
                ws=P, ws_bytes=need)
    for want, kw in ((WS, dict(ws=None)), (WS, dict(ws_bytes=need - 1)), (ALIGN, dict(ws=P + 128))):
        _check(lib, "fp8_scaled_grouped_gemm_blockwise_wgrad", long, want, kw)


# A tile of transposed codes is addressed in 32 bits from its corner.
WIDE = [(LAYOUT, dict(qt=P, recip_t=P, ld_y=1 << 22)), (LAYOUT, dict(qt=P, recip_t=P, q=P, recip=P, ld_q=1 << 24)),
        (LAYOUT, dict(qt=P, recip_t=P, ld_qt=1 << 24))]


@pytest.mark.parametrize("want, kw", WIDE)
def test_strides_of_transposed_tiles(lib, want, kw):
    _check(lib, "fp8bw_moe_gather", GATHER, want, dict(out=_layouts(**kw)))
    _check(lib, "fp8bw_moe_combine_bwd", COMBINE_BWD, want, dict(dy=_layouts(**kw), dweight=None))
    wide = dict(ld_y=512, ld_q=512, rst_kb=512)
    _check(lib, "fp8bw_swiglu_bwd", SWIGLU_BWD, want, dict(dh=_layouts(**{**wide, **kw})))


def test_strides_of_read_tiles(lib):
    qt = _layouts(qt=P, recip_t=P)
    _check(lib, "fp8bw_swiglu_fwd", SWIGLU_FWD, LAYOUT, dict(ld_h=1 << 22, out=qt))
    qt = _layouts(qt=P, recip_t=P, ld_y=512, ld_q=512, rst_kb=512)
    for kw in (dict(ld_h=1 << 22), dict(ld_dy=1 << 22), dict(ld_h=1 << 24, h_recip=P), dict(hr_row=1 << 22, hr_kb=1, h_recip=P),
               dict(act_qt=P, act_recip_t=P, ld_act_qt=1 << 24)):
        _check(lib, "fp8bw_swiglu_bwd", SWIGLU_BWD, LAYOUT, dict(dh=qt, **kw))
