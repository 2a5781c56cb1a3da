"""PyTorch integration of the FP8 blockwise linear: custom ops, autograd and
an nn.Linear counterpart.

The layer above the hot path in the pages' design is a linear module whose
forward and backward quantize and run the blockwise-scaled GEMM
(pytorch/ao PR "integrate torch._scaled_mm into Float8BlockwiseLinear and
add bench script", Summary).  Here that is:

  * three custom ops, ``torch.ops.fp8bw.linear_fwd`` / ``linear_dgrad`` /
    ``linear_wgrad``, each one call of the C ABI (quantizers + GEMM all run
    in libfp8bw.so) with a fake (meta) implementation, so ``torch.compile``
    can trace through them without running them;
  * ``torch.ops.fp8bw.linear``, the forward op with autograd registered:
    its backward calls the dgrad and wgrad ops, each with the recipe the
    pages use for that GEMM (dY 1x128 x W^T 128x128; dY^T 1x128 x X^T 1x128
    along the token axis);
  * ``torch.ops.fp8bw.linear_fwd_save`` / ``linear_bwd``: the same
    computation with X and dY each quantized once per step into both code
    layouts (the forward keeps the X^T codes, the backward quantizes dY
    once and W^T right before the dgrad GEMM), bit-identical to the ops
    above;
  * ``Float8BlockwiseLinear``, a module with ``nn.Linear``'s interface
    (bias-free) that flattens leading dimensions into the token axis and
    trains through the fused-quantization ops;
  * around it, what the rest of a training step needs: ``RMSNorm`` (with the
    residual's addition), ``RMSNormLinear`` (the norm writes the linear's
    operand codes itself), ``linear_cross_entropy`` (a head and its loss
    without the logits) and ``AdamW`` (fp32 or 8-bit states).

Shapes follow the ABI's rules: in_features and out_features multiples of
128 (they are contraction axes in fwd and dgrad) and a token count that is a
multiple of 128 when the weight gradient is needed (its contraction axis).
Everything is bf16.  There is no fallback: without libfp8bw.so the ops raise.
"""

import math
from typing import Optional

import torch

from . import ops


def _check_2d_bf16(*ts):
    for t in ts:
        if t.dim() != 2 or t.dtype != torch.bfloat16:
            raise ValueError("fp8bw linear ops take 2-D bf16 tensors")


@torch.library.custom_op("fp8bw::linear_fwd", mutates_args=())
def linear_fwd(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """Y[M, N] = X[M, K] . W[N, K]^T, X 1x128 and W 128x128 blocks."""
    _check_2d_bf16(x, w)
    return ops.fp8_linear_fwd(x.contiguous(), w.contiguous())


@linear_fwd.register_fake
def _linear_fwd_fake(x, w):
    _check_2d_bf16(x, w)
    return x.new_empty((x.shape[0], w.shape[0]))


@torch.library.custom_op("fp8bw::linear_dgrad", mutates_args=())
def linear_dgrad(dy: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """dX[M, K] = dY[M, N] . W[N, K], dY 1x128 and W^T 128x128 blocks."""
    _check_2d_bf16(dy, w)
    return ops.fp8_linear_dgrad(dy.contiguous(), w.contiguous())


@linear_dgrad.register_fake
def _linear_dgrad_fake(dy, w):
    _check_2d_bf16(dy, w)
    return dy.new_empty((dy.shape[0], w.shape[1]))


@torch.library.custom_op("fp8bw::linear_wgrad", mutates_args=())
def linear_wgrad(dy: torch.Tensor, x: torch.Tensor) -> torch.Tensor:
    """dW[N, K] = dY[M, N]^T . X[M, K], both 1x128 blocks along M."""
    _check_2d_bf16(dy, x)
    return ops.fp8_linear_wgrad(dy.contiguous(), x.contiguous())


@linear_wgrad.register_fake
def _linear_wgrad_fake(dy, x):
    _check_2d_bf16(dy, x)
    return dy.new_empty((dy.shape[1], x.shape[1]))


@torch.library.custom_op("fp8bw::linear", mutates_args=())
def linear(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """Differentiable FP8 blockwise linear: Y = X . W^T (see linear_fwd)."""
    _check_2d_bf16(x, w)
    return ops.fp8_linear_fwd(x.contiguous(), w.contiguous())


@linear.register_fake
def _linear_fake(x, w):
    _check_2d_bf16(x, w)
    return x.new_empty((x.shape[0], w.shape[0]))


def _linear_setup_context(ctx, inputs, output):
    x, w = inputs
    ctx.save_for_backward(x, w)


def _linear_backward(ctx, dy):
    x, w = ctx.saved_tensors
    dy = dy.contiguous()
    dx = torch.ops.fp8bw.linear_dgrad(dy, w) if ctx.needs_input_grad[0] else None
    dw = torch.ops.fp8bw.linear_wgrad(dy, x) if ctx.needs_input_grad[1] else None
    return dx, dw


torch.library.register_autograd("fp8bw::linear", _linear_backward,
                                setup_context=_linear_setup_context)


@torch.library.custom_op("fp8bw::linear_fwd_save", mutates_args=())
def linear_fwd_save(x: torch.Tensor, w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(Y, saved): Y = X . W^T with X quantized once into both code layouts;
    saved holds the X^T codes and scales for linear_bwd (one C-ABI call,
    fp8_linear_fwd_save)."""
    _check_2d_bf16(x, w)
    return ops.fp8_linear_fwd_save(x.contiguous(), w.contiguous())


@linear_fwd_save.register_fake
def _linear_fwd_save_fake(x, w):
    _check_2d_bf16(x, w)
    M, K = x.shape
    N = w.shape[0]
    n = max(ops.linear_saved_bytes(M, N, K), 1)
    return x.new_empty((M, N)), x.new_empty((n,), dtype=torch.uint8)


@torch.library.custom_op("fp8bw::linear_bwd", mutates_args=())
def linear_bwd(dy: torch.Tensor, w: torch.Tensor, saved: torch.Tensor, need_dx: bool,
               need_dw: bool) -> tuple[torch.Tensor, torch.Tensor]:
    """(dX, dW) from dY (quantized once into both layouts), the forward's W
    and the saved buffer of linear_fwd_save; a gradient not asked for comes
    back empty."""
    _check_2d_bf16(dy, w)
    dx, dw = ops.fp8_linear_bwd(dy.contiguous(), w.contiguous(), saved, need_dx, need_dw)
    return (dx if dx is not None else dy.new_empty((0,)),
            dw if dw is not None else dy.new_empty((0,)))


@linear_bwd.register_fake
def _linear_bwd_fake(dy, w, saved, need_dx, need_dw):
    _check_2d_bf16(dy, w)
    M, N = dy.shape
    k = w.shape[1]
    return (dy.new_empty((M, k)) if need_dx else dy.new_empty((0,)),
            dy.new_empty((N, k)) if need_dw else dy.new_empty((0,)))


class _FusedQuantLinear(torch.autograd.Function):
    """Y = X . W^T whose backward uses the X^T codes its forward wrote (X and
    dY each read once per training step)."""

    @staticmethod
    def forward(ctx, x, w):
        y, saved = torch.ops.fp8bw.linear_fwd_save(x, w)
        ctx.save_for_backward(w, saved)
        return y

    @staticmethod
    def backward(ctx, dy):
        w, saved = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        dx, dw = torch.ops.fp8bw.linear_bwd(dy.contiguous(), w, saved, need_dx, need_dw)
        return (dx if need_dx else None), (dw if need_dw else None)


class Float8BlockwiseLinear(torch.nn.Module):
    """Bias-free ``nn.Linear`` counterpart whose forward and backward run the
    FP8 blockwise recipe: y = x W^T with x quantized per 1x128 and W per
    128x128 block; dX and dW as in ``torch.ops.fp8bw.linear``.

    The weight is a bf16 parameter [out_features, in_features] initialized
    as ``nn.Linear`` does (U(+-1/sqrt(in_features))).  Inputs [..., in_features]
    are flattened to [tokens, in_features]."""

    def __init__(self, in_features, out_features, bias=False, device=None, dtype=torch.bfloat16):
        super().__init__()
        if bias:
            raise NotImplementedError("Float8BlockwiseLinear is bias-free")
        if dtype != torch.bfloat16:
            raise ValueError("Float8BlockwiseLinear keeps a bf16 weight")
        if in_features % 128 or out_features % 128:
            raise ValueError("in_features and out_features must be multiples of 128")
        self.in_features = in_features
        self.out_features = out_features
        self.weight = torch.nn.Parameter(
            torch.empty(out_features, in_features, device=device, dtype=dtype))
        self.reset_parameters()

    def reset_parameters(self):
        bound = 1.0 / math.sqrt(self.in_features)
        with torch.no_grad():
            self.weight.uniform_(-bound, bound)

    @classmethod
    def from_linear(cls, lin):
        """The same layer from a bias-free ``nn.Linear`` (weight cast to bf16)."""
        if lin.bias is not None:
            raise NotImplementedError("Float8BlockwiseLinear is bias-free")
        m = cls(lin.in_features, lin.out_features, device=lin.weight.device)
        with torch.no_grad():
            m.weight.copy_(lin.weight.to(torch.bfloat16))
        return m

    def forward(self, x):
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features)
        if torch.is_grad_enabled() and (x.requires_grad or self.weight.requires_grad):
            # Training: quantize X once into both layouts and keep the
            # transposed fp8 codes (half the bytes of the bf16 X) for backward.
            # The weight gradient contracts over the tokens in 1x128 blocks,
            # so their count must be a multiple of 128; say so here rather
            # than in the backward.
            if x2.shape[0] % 128:
                raise ValueError(f"training needs the token count ({x2.shape[0]}) to be a multiple "
                                 "of 128: the weight gradient contracts over tokens in blocks of 128")
            y = _FusedQuantLinear.apply(x2, self.weight)
        else:
            y = torch.ops.fp8bw.linear_fwd(x2, self.weight)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self):
        return f"in_features={self.in_features}, out_features={self.out_features}, bias=False"


# ---------------------------------------------------------------------------
# RMS norm.


def _empty(like, dtype=None):
    return like.new_empty((0,), dtype=dtype)


def _aligned(t):
    """t where it is laid out as the kernels read it (16-byte aligned rows of
    unit column stride), else a copy that is."""
    if t is None or t.numel() == 0:
        return t
    rows_fit = t.dim() < 2 or t.shape[0] == 1 or (t.stride(0) >= t.shape[1] and t.stride(0) % 8 == 0)
    if t.data_ptr() % 16 == 0 and t.stride(-1) == 1 and rows_fit:
        return t
    return t.clone(memory_format=torch.contiguous_format)


@torch.library.custom_op("fp8bw::rms_norm_fwd", mutates_args=())
def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor],
                 eps: float) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y, s, rstd) of ops.rms_norm_fwd; s comes back empty without a
    residual (it is x)."""
    o = ops.rms_norm_fwd(_aligned(x), _aligned(weight), residual=_aligned(residual), eps=eps)
    return o.y, (_empty(x) if residual is None else o.s), o.rstd


@rms_norm_fwd.register_fake
def _rms_norm_fwd_fake(x, weight, residual, eps):
    _check_2d_bf16(x)
    rows, cols = x.shape
    return (x.new_empty((rows, cols)), _empty(x) if residual is None else x.new_empty((rows, cols)),
            x.new_empty((rows,), dtype=torch.float32))


@torch.library.custom_op("fp8bw::rms_norm_bwd", mutates_args=())
def rms_norm_bwd(dy: torch.Tensor, s: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                 dres: Optional[torch.Tensor]) -> tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight) of ops.rms_norm_bwd."""
    return ops.rms_norm_bwd(_aligned(dy), _aligned(s), rstd, _aligned(weight), _aligned(dres))


@rms_norm_bwd.register_fake
def _rms_norm_bwd_fake(dy, s, rstd, weight, dres):
    return dy.new_empty(dy.shape), torch.empty_like(weight)


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, s, rstd = torch.ops.fp8bw.rms_norm_fwd(x, weight, residual, eps)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)   # an unused sum costs no reading of zeros
        ctx.save_for_backward(x if residual is None else s, rstd, weight)
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, rstd, weight = ctx.saved_tensors
        dres = ds if ctx.has_residual else None
        if dy is None:
            return dres, dres, None, None
        dx, dweight = torch.ops.fp8bw.rms_norm_bwd(dy, s, rstd, weight, dres)
        return dx, (dx if ctx.has_residual else None), dweight, None


class RMSNorm(torch.nn.Module):
    """Root-mean-square norm of [..., features] bf16 with a learned weight.
    ``norm(x)`` returns y; ``norm(x, residual)`` returns (y, x + residual), the
    sum in bf16 being the next residual."""

    def __init__(self, features, eps=1e-6, device=None, dtype=torch.bfloat16):
        super().__init__()
        if features % 16:
            raise ValueError("features must be a multiple of 16")
        self.features, self.eps = features, eps
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))

    def forward(self, x, residual=None):
        shape = x.shape
        x2 = x.reshape(-1, self.features)
        r2 = None if residual is None else residual.reshape(-1, self.features)
        y, s = _RMSNorm.apply(x2, r2, self.weight, self.eps)
        return y.reshape(shape) if residual is None else (y.reshape(shape), s.reshape(shape))

    def extra_repr(self):
        return f"{self.features}, eps={self.eps}"


# ---------------------------------------------------------------------------
# RMS norm and FP8 linear in one: the norm writes the E4M3 codes of the GEMM's
# operand (and, training, of its transpose), so the bf16 normed activation
# never exists.

@torch.library.custom_op("fp8bw::norm_linear_fwd", mutates_args=())
def norm_linear_fwd(x: torch.Tensor, residual: Optional[torch.Tensor], norm_weight: torch.Tensor,
                    w: torch.Tensor, eps: float, train: bool
                    ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(Y, s, rstd, qt, recip_t): Y = norm(x + residual) . W^T; s empty without
    a residual, qt and recip_t (for W's gradient) empty unless train."""
    _check_2d_bf16(x, w)
    o = ops.rms_norm_fwd(_aligned(x), _aligned(norm_weight), residual=_aligned(residual), eps=eps, y=False,
                         q=True, qt=train)
    wq, wr = ops.fp8_blockwise_quant(_aligned(w), "128x128")
    out = ops.fp8_scaled_gemm_blockwise(o.q, o.recip, wq, wr)
    return (out, _empty(x) if residual is None else o.s, o.rstd,
            o.qt if train else _empty(x, torch.uint8),
            o.recip_t if train else _empty(x, torch.float32))


@norm_linear_fwd.register_fake
def _norm_linear_fwd_fake(x, residual, norm_weight, w, eps, train):
    _check_2d_bf16(x, w)
    M, K = x.shape
    return (x.new_empty((M, w.shape[0])), _empty(x) if residual is None else x.new_empty((M, K)),
            x.new_empty((M,), dtype=torch.float32),
            x.new_empty((K, M), dtype=torch.uint8) if train else _empty(x, torch.uint8),
            x.new_empty(((M + 127) // 128, K), dtype=torch.float32).t() if train
            else _empty(x, torch.float32))


@torch.library.custom_op("fp8bw::norm_linear_bwd", mutates_args=())
def norm_linear_bwd(dy: torch.Tensor, ds: Optional[torch.Tensor], s: torch.Tensor,
                    rstd: torch.Tensor, norm_weight: torch.Tensor, w: torch.Tensor,
                    qt: torch.Tensor, recip_t: torch.Tensor, need_dx: bool = True,
                    need_dw: bool = True) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dx, dnorm_weight, dW): dgrad and wgrad GEMMs on the linear's recipe,
    then the norm's backward on the dgrad.  Without need_dx (dx and
    dnorm_weight) or need_dw those come back empty."""
    dy = _aligned(dy)
    if need_dx and need_dw:
        dyq, dyr, dytq, dytr = ops.fp8_blockwise_quant_dual(dy, "1x128")
    elif need_dx:
        dyq, dyr = ops.fp8_blockwise_quant(dy, "1x128")
    elif need_dw:
        dytq, dytr = ops.fp8_blockwise_quant(dy, "1x128", transpose=True)
    dx = dnorm = dw = None
    if need_dx:
        wtq, wtr = ops.fp8_blockwise_quant(_aligned(w), "128x128", transpose=True)
        dx, dnorm = ops.rms_norm_bwd(ops.fp8_scaled_gemm_blockwise(dyq, dyr, wtq, wtr), _aligned(s), rstd,
                                     _aligned(norm_weight), _aligned(ds))
    if need_dw:
        dw = ops.fp8_scaled_gemm_blockwise(dytq, dytr, qt, recip_t, b_block="1x128")
    return (_empty(s) if dx is None else dx, _empty(norm_weight) if dnorm is None else dnorm,
            _empty(w) if dw is None else dw)


@norm_linear_bwd.register_fake
def _norm_linear_bwd_fake(dy, ds, s, rstd, norm_weight, w, qt, recip_t, need_dx=True, need_dw=True):
    return (s.new_empty(s.shape) if need_dx else _empty(s),
            torch.empty_like(norm_weight) if need_dx else _empty(norm_weight),
            w.new_empty(w.shape) if need_dw else _empty(w))


class _RMSNormLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, norm_weight, w, eps):
        y, s, rstd, qt, recip_t = torch.ops.fp8bw.norm_linear_fwd(x, residual, norm_weight, w, eps,
                                                                  ctx.needs_input_grad[3])
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if residual is None else s, rstd, norm_weight, w, qt, recip_t)
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, rstd, norm_weight, w, qt, recip_t = ctx.saved_tensors
        dres = ds if ctx.has_residual else None
        if dy is None:
            return dres, dres, None, None, None
        need_dx, need_dw = any(ctx.needs_input_grad[:3]), ctx.needs_input_grad[3]
        dx, dnorm, dw = torch.ops.fp8bw.norm_linear_bwd(dy, dres, s, rstd, norm_weight, w,
                                                        qt, recip_t, need_dx, need_dw)
        if not need_dx:
            dx = dnorm = None
        return (dx, (dx if ctx.has_residual else None), dnorm,
                dw if need_dw else None, None)


class RMSNormLinear(torch.nn.Module):
    """``Float8BlockwiseLinear(RMSNorm(x))`` with the norm writing the linear's
    FP8 operand.  ``m(x)`` returns y; ``m(x, residual)`` returns (y, x +
    residual).  Training needs a token count that is a multiple of 128."""

    def __init__(self, in_features, out_features, eps=1e-6, device=None):
        super().__init__()
        self.norm = RMSNorm(in_features, eps, device=device)
        self.linear = Float8BlockwiseLinear(in_features, out_features, device=device)

    def forward(self, x, residual=None):
        lin = self.linear
        x2 = x.reshape(-1, lin.in_features)
        r2 = None if residual is None else residual.reshape(-1, lin.in_features)
        args = (x2, r2, self.norm.weight, lin.weight)
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in args):
            if x2.shape[0] % 128:
                raise ValueError(f"training needs the token count ({x2.shape[0]}) to be a multiple of "
                                 "128: the weight gradient contracts over tokens in blocks of 128")
            y, s = _RMSNormLinear.apply(*args, self.norm.eps)
        else:
            y, s = torch.ops.fp8bw.norm_linear_fwd(*args, self.norm.eps, False)[:2]
        y = y.reshape(*x.shape[:-1], lin.out_features)
        return y if residual is None else (y, s.reshape(x.shape))


# ---------------------------------------------------------------------------
# Cross entropy of a linear head.

@torch.library.custom_op("fp8bw::linear_xent_fwd", mutates_args=())
def linear_xent_fwd(h: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                    ignore_index: int) -> tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse) per token of ops.linear_xent_fwd."""
    return ops.linear_xent_fwd(_aligned(h), _aligned(w), target, ignore_index)


@linear_xent_fwd.register_fake
def _linear_xent_fwd_fake(h, w, target, ignore_index):
    _check_2d_bf16(h, w)
    return tuple(h.new_empty((h.shape[0],), dtype=torch.float32) for _ in range(2))


@torch.library.custom_op("fp8bw::linear_xent_bwd", mutates_args=())
def linear_xent_bwd(dloss: torch.Tensor, h: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                    lse: torch.Tensor, ignore_index: int, need_dh: bool, need_dw: bool,
                    loss: Optional[torch.Tensor] = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(dh, dw) of ops.linear_xent_bwd; one not asked for comes back empty."""
    dh, dw = ops.linear_xent_bwd(dloss, _aligned(h), _aligned(w), target, lse, ignore_index, need_dh,
                                 need_dw, loss)
    return (_empty(h) if dh is None else dh), (_empty(w) if dw is None else dw)


@linear_xent_bwd.register_fake
def _linear_xent_bwd_fake(dloss, h, w, target, lse, ignore_index, need_dh, need_dw, loss=None):
    return (h.new_empty(h.shape) if need_dh else _empty(h),
            w.new_empty(w.shape) if need_dw else _empty(w))


class _LinearXent(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, target, ignore_index, exposed):
        loss, lse = torch.ops.fp8bw.linear_xent_fwd(h, w, target, ignore_index)
        ctx.ignore_index = ignore_index
        # the backward's own losses, where the caller gets these and may change them
        ctx.save_for_backward(h, w, target, lse,
                              loss.clone() if exposed and any(ctx.needs_input_grad) else loss)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        h, w, target, lse, loss = ctx.saved_tensors
        need = ctx.needs_input_grad[:2]
        dh, dw = torch.ops.fp8bw.linear_xent_bwd(dloss.contiguous(), h, w, target, lse,
                                                 ctx.ignore_index, *need, loss)
        return (dh if need[0] else None), (dw if need[1] else None), None, None, None


def linear_cross_entropy(h, w, target, ignore_index=-100, reduction="mean"):
    """Cross entropy of logits h . w^T (never kept) against target: h bf16
    [..., K], w bf16 [V, K], target int64 [...].  reduction as in
    ``F.cross_entropy``: "mean" over the tokens that count (NaN if none
    does), "sum" or "none"."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError(f"unknown reduction {reduction!r}")
    flat = target.reshape(-1).contiguous()
    loss = _LinearXent.apply(h.reshape(-1, h.shape[-1]), w, flat, ignore_index, reduction == "none")
    if reduction == "none":
        return loss.reshape(target.shape)
    if reduction == "sum":
        return loss.sum()
    return loss.sum() / (flat != ignore_index).sum()


# ---------------------------------------------------------------------------
# Optimizer.

class AdamW(torch.optim.Optimizer):
    """AdamW whose step is one call of ``fp8bw_adamw_step`` per group.

    state_bits: 32, or 8 for E4M3 codes with a scale per 128 elements (2.06
    bytes of state per parameter instead of 8).  master_weights: fp32 copies
    behind bf16 parameters.  stochastic: round codes, and bf16 parameters
    without a master, up or down at random by a hash of (seed, step, tensor,
    element), a tensor being known by its place among the parameters of all
    groups; default: wherever something is so held.  Optimizers that train side
    by side take different seeds.  ``step(grad_scale=t)`` multiplies every
    gradient by the one-element fp32 tensor t."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, state_bits=32,
                 master_weights=False, stochastic=True, seed=0):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if lr < 0 or eps < 0 or weight_decay < 0 or not all(0 <= b < 1 for b in betas):
            raise ValueError("lr, eps and weight_decay must be >= 0 and betas in [0, 1)")
        self.state_bits, self.master_weights = state_bits, master_weights
        self.stochastic, self.seed = stochastic, seed
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))

    def _new_state(self, p):
        st = {"step": 0}
        n = ops.adamw_scales(p.numel())
        if self.state_bits == 8:
            for k in ("exp_avg", "exp_avg_root"):
                st[k] = torch.zeros(p.numel(), dtype=torch.uint8, device=p.device)
                st[k + "_scale"] = torch.ones(n, dtype=torch.float32, device=p.device)
        else:
            st["exp_avg"] = torch.zeros_like(p, dtype=torch.float32, memory_format=torch.contiguous_format)
            st["exp_avg_sq"] = torch.zeros_like(st["exp_avg"])
        if self.master_weights and p.dtype == torch.bfloat16:
            st["master"] = p.detach().float().contiguous()
        return st

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        first = 0
        for group in self.param_groups:
            by_step = {}
            for ordinal, p in enumerate(group["params"], first):
                if p.grad is None:
                    continue
                if not self.state[p]:
                    self.state[p].update(self._new_state(p))
                st = self.state[p]
                by_step.setdefault((p.device, st["step"] + 1), []).append((p, st, ordinal))
            first += len(group["params"])
            for (_, step), tensors in by_step.items():
                self._step_group(group, step, tensors, grad_scale)
        return loss

    def _step_group(self, group, step, tensors, grad_scale):
        params, states, ordinals = zip(*tensors)
        if ordinals == tuple(range(len(ordinals))):
            ordinals = None   # their places in the lists
        eight = self.state_bits == 8
        second = "exp_avg_root" if eight else "exp_avg_sq"
        ops.adamw_step(params, [p.grad.contiguous() for p in params],
                       [st["exp_avg"] for st in states], [st[second] for st in states], step=step,
                       lr=group["lr"], beta1=group["betas"][0], beta2=group["betas"][1],
                       eps=group["eps"], weight_decay=group["weight_decay"],
                       exp_avg_scales=[st["exp_avg_scale"] for st in states] if eight else None,
                       root_scales=[st["exp_avg_root_scale"] for st in states] if eight else None,
                       masters=[st.get("master") for st in states], grad_scale=grad_scale,
                       seed=(self.seed + 0x9E3779B97F4A7C15 * step) & 0xFFFFFFFFFFFFFFFF
                       if self.stochastic else None, ordinals=ordinals)
        for st in states:
            st["step"] = step

    def load_state_dict(self, state_dict):
        """As torch's, but states keep their types (torch casts floating
        parameters' states to the parameter's type, which codes do not survive).
        States must be of this optimizer's state_bits; masters that the
        checkpoint lacks are made from the parameters."""
        for st in state_dict["state"].values():
            if st and ("exp_avg_root" in st) != (self.state_bits == 8):
                raise ValueError(f"the checkpoint's states do not have state_bits={self.state_bits}")
        super().load_state_dict(state_dict)
        saved = [i for g in state_dict["param_groups"] for i in g["params"]]
        mine = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(saved, mine):
            for k, v in state_dict["state"].get(i, {}).items():
                self.state[p][k] = v.detach().clone().to(p.device) if isinstance(v, torch.Tensor) else v
            if self.state.get(p) and self.master_weights and p.dtype == torch.bfloat16:
                self.state[p].setdefault("master", p.detach().float().contiguous())
