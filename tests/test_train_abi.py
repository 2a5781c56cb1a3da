"""Refusals of the norm, cross entropy and AdamW entry points, without a GPU:
every invalid argument is rejected on the host before any HIP call."""

import ctypes

import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from blockwise_scaled_fp8_amd import _lib

OK, NULL, SHAPE, LAYOUT, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5, 6
P = 0x10000  # a 256-byte aligned fake device address; never dereferenced here
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    return fp8.load_library()


def _norm_fwd(lib, **kw):
    a = dict(x=P, ld_x=256, residual=None, ld_res=256, weight=P, weight_dtype=0, eps=1e-6, rows=32, cols=256,
             sum=None, ld_sum=256, rstd=P, y=P, ld_y=256, q=None, ld_q=256, recip=None, rs_row=1, rs_kb=32,
             qt=None, ld_qt=32, recip_t=None, rst_row=1, rst_kb=256, stream=None)
    a.update(kw)
    return lib.fp8bw_rms_norm_fwd(*a.values())


@pytest.mark.parametrize("want, kw", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=250)), (SHAPE, dict(cols=16400)), (SHAPE, dict(rows=1 << 22)),
    (UNSUP, dict(weight_dtype=2)), (UNSUP, dict(eps=-1.0)), (UNSUP, dict(eps=float("nan"))),
    (NULL, dict(x=None)), (NULL, dict(weight=None)), (NULL, dict(rstd=None)), (NULL, dict(residual=P)),
    (ALIGN, dict(x=P + 8)), (ALIGN, dict(weight=P + 4)), (ALIGN, dict(rstd=P + 2)), (ALIGN, dict(y=P + 8)),
    (LAYOUT, dict(ld_x=240)), (LAYOUT, dict(ld_x=260)), (LAYOUT, dict(ld_y=BIG)), (LAYOUT, dict(ld_x=-8)),
    (LAYOUT, dict(residual=P, sum=P, ld_sum=512)),
    (NULL, dict(q=P)), (ALIGN, dict(q=P + 8, recip=P)), (LAYOUT, dict(q=P, recip=P, ld_q=264)),
    (LAYOUT, dict(q=P, recip=P, rs_kb=16)), (LAYOUT, dict(q=P, recip=P, rs_row=-1)),
    (SHAPE, dict(qt=P, recip_t=P, rows=30)), (LAYOUT, dict(qt=P, recip_t=P, ld_qt=16)),
    (LAYOUT, dict(qt=P, recip_t=P, rst_row=0)),
    (OK, dict(rows=0, x=None, weight=None, rstd=None, y=None)), (OK, dict(cols=0, x=None))])
def test_norm_fwd(lib, want, kw):
    assert _norm_fwd(lib, **kw) == want
    assert bool(lib.fp8bw_last_error()) == (want != OK)


def test_norm_bwd(lib):
    need = lib.fp8bw_rms_norm_bwd_ws_bytes(32, 256)
    assert need > 0 and lib.fp8bw_rms_norm_bwd_ws_bytes(0, 256) == 0
    assert lib.fp8bw_rms_norm_bwd_ws_bytes(BIG, 256) == 0

    def call(**kw):
        a = dict(dy=P, ld_dy=256, s=P, ld_s=256, rstd=P, weight=P, weight_dtype=1, dres=None, ld_dres=0, rows=32,
                 cols=256, dx=P, ld_dx=256, dweight=P, ws=P, ws_bytes=need, stream=None)
        a.update(kw)
        return lib.fp8bw_rms_norm_bwd(*a.values())
    for want, kw in ((SHAPE, dict(cols=8)), (NULL, dict(dy=None)), (NULL, dict(dweight=None)), (NULL, dict(dx=None)),
                     (LAYOUT, dict(ld_s=128)), (ALIGN, dict(dres=P + 2)), (LAYOUT, dict(dres=P, ld_dres=8)),
                     (WS, dict(ws_bytes=need - 1)), (WS, dict(ws=None)), (ALIGN, dict(ws=P + 4)),
                     (UNSUP, dict(weight_dtype=-1)), (OK, dict(rows=0, dy=None, dx=None))):
        assert call(**kw) == want, kw


def test_xent(lib):
    f, b = lib.fp8bw_linear_xent_ws_bytes(33, 1000, 128, 0), lib.fp8bw_linear_xent_ws_bytes(33, 1000, 128, 1)
    assert f >= 33 * 4 * 8 and b >= 64 * 1000 * 2
    for T, V, K in ((0, 10, 64), (10, 0, 64), (10, 10, 65), (-1, 10, 64), (BIG, 10, 64), (10, BIG, 64), (10, 10, BIG)):
        assert lib.fp8bw_linear_xent_ws_bytes(T, V, K, 1) == 0
    # one piece of the vocabulary, however long it is
    assert lib.fp8bw_linear_xent_ws_bytes(8192, 1 << 20, 4096, 1) < (1 << 29)

    def fwd(**kw):
        a = dict(h=P, ld_h=128, w=P, ld_w=128, target=P, ignore=-100, T=33, V=1000, K=128, loss=P, lse=P, ws=P,
                 ws_bytes=f, stream=None)
        a.update(kw)
        return lib.fp8bw_linear_xent_fwd(*a.values())

    def bwd(**kw):
        a = dict(dloss=P, h=P, ld_h=128, w=P, ld_w=128, target=P, ignore=-100, lse=P, T=33, V=1000, K=128, dh=P,
                 ld_dh=128, dw=P, ld_dw=128, ws=P, ws_bytes=b, stream=None)
        a.update(kw)
        return lib.fp8bw_linear_xent_bwd(*a.values())
    for call in (fwd, bwd):
        for want, kw in ((SHAPE, dict(K=96)), (SHAPE, dict(K=0)), (SHAPE, dict(T=-1)), (SHAPE, dict(V=0)),
                         (SHAPE, dict(T=1 << 24, V=1 << 28)), (NULL, dict(h=None)), (NULL, dict(w=None)),
                         (NULL, dict(target=None)), (NULL, dict(lse=None)), (ALIGN, dict(target=P + 4)),
                         (ALIGN, dict(w=P + 2)), (LAYOUT, dict(ld_h=120)), (LAYOUT, dict(ld_w=132)),
                         (LAYOUT, dict(ld_w=1 << 23)), (WS, dict(ws=None)), (WS, dict(ws_bytes=8)),
                         (ALIGN, dict(ws=P + 16))):
            assert call(**kw) == want, (call, kw)
    assert fwd(T=0, h=None, target=None) == OK and bwd(T=0, dw=None, h=None) == OK
    assert fwd(loss=None) == NULL and bwd(dloss=None) == NULL
    assert bwd(ld_dw=64) == LAYOUT and bwd(dh=P + 8) == ALIGN
    assert bwd(dh=None, dw=None) == OK


def _adamw(lib, tensors=1, count=None, state=0, step=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, scale=None, **kw):
    arr = (_lib.AdamwTensor * max(tensors, 1))()
    for t in arr:
        t.param = t.grad = t.exp_avg = t.exp_avg_sq = P
        t.numel, t.param_dtype, t.grad_dtype = 10, 0, 1
        if state == 1:
            t.exp_avg_scale = t.root_scale = P
    for k, v in kw.items():
        setattr(arr[tensors - 1], k, v)
    return lib.fp8bw_adamw_step(arr, tensors if count is None else count, state, step, lr, b1, b2, eps, wd, scale, 0, 0, None)


@pytest.mark.parametrize("want, kw", [
    (SHAPE, dict(count=-1)), (OK, dict(count=0)), (UNSUP, dict(state=2)), (SHAPE, dict(step=0)),
    (UNSUP, dict(lr=-1.0)), (UNSUP, dict(lr=float("inf"))), (UNSUP, dict(b1=1.0)), (UNSUP, dict(b2=-0.1)),
    (UNSUP, dict(eps=float("nan"))), (UNSUP, dict(wd=-1.0)), (ALIGN, dict(scale=P + 1)),
    (NULL, dict(param=None)), (NULL, dict(tensors=3, grad=None)), (NULL, dict(exp_avg=None)), (NULL, dict(exp_avg_sq=None)),
    (NULL, dict(state=1, root_scale=None)), (UNSUP, dict(exp_avg_scale=P)), (SHAPE, dict(numel=-1)),
    (SHAPE, dict(numel=BIG)), (UNSUP, dict(param_dtype=3)), (UNSUP, dict(grad_dtype=-1)),
    (UNSUP, dict(param_dtype=1, master=P)), (ALIGN, dict(param=P + 1)), (ALIGN, dict(grad=P + 2)),
    (ALIGN, dict(master=P + 2)), (ALIGN, dict(exp_avg=P + 2)), (OK, dict(numel=0, param=None, grad=None))])
def test_adamw(lib, want, kw):
    assert _adamw(lib, **kw) == want


def test_adamw_struct_is_the_headers():
    """7 pointers, a length and two enums."""
    assert ctypes.sizeof(_lib.AdamwTensor) == 7 * 8 + 8 + 2 * 4


def test_binding_refuses_host_tensors_and_wrong_types():
    x, w = torch.zeros(16, 128, dtype=torch.bfloat16), torch.zeros(128)
    t = torch.zeros(16, dtype=torch.int64)
    f = torch.zeros(16)
    for call in (lambda: fp8.rms_norm_fwd(x, w), lambda: fp8.rms_norm_bwd(x, x, f, w),
                 lambda: fp8.linear_xent_fwd(x, x, t), lambda: fp8.linear_xent_bwd(f, x, x, t, f),
                 lambda: fp8.adamw_step([f], [f], [f], [f], step=1, lr=0.1)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="8-bit"):
        fp8.adamw_step([f], [f], [f.byte()], [f.byte()], step=1, lr=0.1)
    with pytest.raises(ValueError, match="grads"):
        fp8.adamw_step([f], [f, f], [f], [f], step=1, lr=0.1)
    assert fp8.adamw_step([], [], [], [], step=1, lr=0.1) is None
    with pytest.raises(ValueError, match="reduction"):
        fp8.linear_cross_entropy(x, x, t, reduction="all")
    with pytest.raises(ValueError, match="state_bits"):
        fp8.AdamW([torch.nn.Parameter(f)], state_bits=4)


def test_modules_on_meta_tensors():
    """Shapes through forward and backward without running anything."""
    x = torch.empty(2, 128, 256, dtype=torch.bfloat16, device="meta", requires_grad=True)
    r = torch.empty_like(x).requires_grad_()
    norm, lin = fp8.RMSNorm(256, device="meta"), fp8.RMSNormLinear(256, 384, device="meta")
    y, s = norm(x, r)
    z, s2 = lin(y, s)
    assert y.shape == s.shape == s2.shape == x.shape and z.shape == (2, 128, 384)
    head = torch.empty(1000, 384, dtype=torch.bfloat16, device="meta", requires_grad=True)
    target = torch.empty(2, 128, dtype=torch.int64, device="meta")
    (fp8.linear_cross_entropy(z, head, target) + s2.float().sum()).backward()
    for t in (x, r, head, norm.weight, lin.norm.weight, lin.linear.weight):
        assert t.grad.shape == t.shape
    with pytest.raises(ValueError, match="multiple of 128"):
        lin(torch.empty(50, 256, dtype=torch.bfloat16, device="meta"))
    with torch.no_grad():
        assert lin(torch.empty(50, 256, dtype=torch.bfloat16, device="meta")).shape == (50, 384)
    assert norm(x).shape == x.shape


def test_compile_traces_norm_linear_and_loss():
    class Net(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.lin = fp8.RMSNormLinear(128, 256, device="meta")
            self.head = torch.nn.Parameter(torch.empty(500, 256, dtype=torch.bfloat16, device="meta"))

        def forward(self, x, t):
            return fp8.linear_cross_entropy(self.lin(x), self.head, t, reduction="sum")
    x = torch.empty(128, 128, dtype=torch.bfloat16, device="meta", requires_grad=True)
    t = torch.empty(128, dtype=torch.int64, device="meta")
    torch.compile(Net(), backend="aot_eager", fullgraph=True)(x, t).backward()
    assert x.grad.shape == x.shape
