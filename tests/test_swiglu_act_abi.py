"""swiglu_bwd asked for the activation's transposed codes alone takes no dy; asked
for any gradient it does (no GPU: refusals on the host)."""

import ctypes

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from blockwise_scaled_fp8_amd import _lib

OK, NULL, SHAPE, LAYOUT, ALIGN = 0, 1, 2, 3, 4
P = 0x10000


def _dh(**kw):
    a = dict(y=None, ld_y=512, q=None, ld_q=512, recip=None, rs_row=1, rs_kb=64, qt=None, ld_qt=64, recip_t=None, rst_row=1,
             rst_kb=512)
    a.update(kw)
    return ctypes.byref(_lib.Layouts(*a.values()))


BASE = dict(dy=None, ld_dy=0, h=P, ld_h=512, h_recip=None, hr_row=1, hr_kb=64, rows=64, ffn=256, dh=_dh(), act_qt=P,
            ld_act_qt=64, act_recip_t=P, art_row=1, art_kb=256, stream=None)


@pytest.mark.parametrize("want, kw", [
    (NULL, dict(dh=_dh(y=P))), (NULL, dict(dh=_dh(q=P, recip=P))), (NULL, dict(dh=_dh(qt=P, recip_t=P))),
    (NULL, dict(dh=None)), (NULL, dict(h=None)), (NULL, dict(act_recip_t=None)), (LAYOUT, dict(ld_act_qt=48)),
    (LAYOUT, dict(ld_h=1 << 22)), (LAYOUT, dict(ld_h=1 << 24, h_recip=P)), (SHAPE, dict(rows=60)),
    (ALIGN, dict(dy=P + 8, ld_dy=256)), (LAYOUT, dict(dy=P, ld_dy=248)), (OK, dict(act_qt=None)), (OK, dict(rows=0)),
    (OK, dict(ffn=0))])
def test_refusals(want, kw):
    lib = fp8.load_library()
    assert set(kw) <= set(BASE)
    assert lib.fp8bw_swiglu_bwd(*{**BASE, **kw}.values()) == want
    assert bool(lib.fp8bw_last_error()) == (want != OK)


def test_the_binding_asks_for_dy_where_a_gradient_is_wanted():
    h = torch.zeros(16, 64, dtype=torch.bfloat16)
    for kw in (dict(), dict(dh=False, q=True, act_qt=True), dict(dh=False, qt=True), dict(dh=False, act_qt=True)):
        with pytest.raises(ValueError, match="HIP"):
            fp8.swiglu_bwd(None, h, **kw)
