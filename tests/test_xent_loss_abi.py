"""Refusals of the cross entropy's backward with losses, without a GPU."""

import torch

import blockwise_scaled_fp8_amd as fp8

P = 0x10000  # a 256-byte aligned fake device address; never dereferenced here


def test_backward_with_losses():
    lib = fp8.load_library()
    need = lib.fp8bw_linear_xent_ws_bytes(33, 1000, 128, 1)

    def bwd(**kw):
        a = dict(dloss=P, h=P, ld_h=128, w=P, ld_w=128, target=P, ignore=-100, lse=P, loss=P, T=33, V=1000, K=128,
                 dh=P, ld_dh=128, dw=P, ld_dw=128, ws=P, ws_bytes=need, stream=None)
        a.update(kw)
        return lib.fp8bw_linear_xent_bwd_loss(*a.values())
    # FP8BW_ERR_ALIGN, _NULL, _SHAPE, _LAYOUT, _WORKSPACE; nothing to do
    for want, kw in ((4, dict(loss=P + 2)), (1, dict(lse=None)), (1, dict(dloss=None)), (2, dict(V=0)),
                     (3, dict(ld_h=64)), (6, dict(ws_bytes=need - 1)), (0, dict(T=0, dw=None, loss=None)),
                     (0, dict(dh=None, dw=None, loss=None))):
        assert bwd(**kw) == want, kw


def test_fake_takes_losses():
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        h, w = torch.empty(8, 64, dtype=torch.bfloat16), torch.empty(100, 64, dtype=torch.bfloat16)
        f, t = torch.empty(8), torch.empty(8, dtype=torch.int64)
        for loss in ((), (f,)):
            dh, dw = torch.ops.fp8bw.linear_xent_bwd(f, h, w, t, f, -100, True, False, *loss)
            assert dh.shape == (8, 64) and dw.numel() == 0
