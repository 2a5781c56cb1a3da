"""Thin torch-facing binding of the C ABI: the same entry-point names as
include/fp8bw.h.  Each function only checks tensor placement, allocates its
outputs with torch (device memory is plumbing), passes raw pointers, sizes and
the current HIP stream, and raises FP8BWError on a non-OK status.  Every step
of the computation runs in the HIP kernels of libfp8bw.so."""

import array
import functools
from typing import NamedTuple, Optional

import torch

from ._lib import AdamwTensor, Layouts, check, load_library

BLOCKS = {"1x128": 0, "128x128": 1}
OUT_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def _stream(t):
    # the raw handle of torch's current stream on t's device (the direct C
    # accessor: torch.cuda.current_stream(device) costs microseconds per call)
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _need_cuda(*ts):
    for t in ts:
        if not (isinstance(t, torch.Tensor) and t.is_cuda):
            raise ValueError("fp8bw ops take CUDA (HIP) tensors")


def _on_tensor_device(fn):
    """Every tensor argument (inputs and caller-provided outputs or
    workspace) must be a HIP tensor on one device; that device is made
    current for the call, so the library's launches, its per-device queries
    and the stream all refer to the device that holds the data."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        dev = None
        for t in list(args) + list(kwargs.values()):
            if not isinstance(t, torch.Tensor):
                continue
            if not t.is_cuda:
                raise ValueError("fp8bw ops take CUDA (HIP) tensors")
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"fp8bw ops take tensors on one device ({dev} and {t.device} given)")
        if dev is None or dev.index == torch._C._cuda_getDevice():
            return fn(*args, **kwargs)
        with torch.cuda.device(dev):
            return fn(*args, **kwargs)
    return wrapper


def _rowmajor(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")


def _cdiv(a, b):
    return (a + b - 1) // b


def scale_grid(rows, cols, block, transpose):
    """Logical shape (ni, nj) of the reciprocal-scale tensor."""
    if block == "1x128":
        return (cols, _cdiv(rows, 128)) if transpose else (rows, _cdiv(cols, 128))
    return (_cdiv(cols, 128), _cdiv(rows, 128)) if transpose else (_cdiv(rows, 128), _cdiv(cols, 128))


def colmajor_empty(ni, nj, device):
    """fp32 [ni, nj] with column-major strides (1, ni)."""
    return torch.empty((nj, max(ni, 1)), dtype=torch.float32, device=device)[:, :ni].t()


def _check_codes(a, b, K):
    for t in (a, b):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise ValueError("GEMM operands are E4M3 codes (uint8 or float8_e4m3fn)")
    if b.shape[1] != K:
        raise ValueError(f"b has K={b.shape[1]}, a has K={K}")


def _check_shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


CODE_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def _check_codes_out(t, shape, name):
    """A caller-provided code buffer: E4M3 bytes, row-major rows."""
    _check_shape(t, shape, name)
    if t.dtype not in CODE_DTYPES:
        raise ValueError(f"{name} must be uint8 or float8_e4m3fn, got {t.dtype}")
    _rowmajor(t, name)


def _check_scales(t, shape, name):
    """fp32 reciprocal scales of a given logical shape (any strides; the
    library checks that they do not overlap)."""
    _check_shape(t, shape, name)
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32, got {t.dtype}")


def _check_out(t, shape, name="out"):
    _check_shape(t, shape, name)
    if t.dtype not in OUT_DTYPES:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    _rowmajor(t, name)


@_on_tensor_device
def fp8_blockwise_quant(x, block="1x128", transpose=False, q=None, recip=None):
    """Quantize bf16 x[rows, cols] to E4M3 codes with per-block reciprocal scales.

    Returns (q, recip): q uint8 [rows, cols] (or [cols, rows] with transpose),
    recip fp32 [ni, nj] (column-major unless a tensor is passed in)."""
    lib = load_library()
    _need_cuda(x)
    _rowmajor(x, "x")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    rows, cols = x.shape
    qshape = (cols, rows) if transpose else (rows, cols)
    if q is None:
        q = torch.empty(qshape, dtype=torch.uint8, device=x.device)
    _check_codes_out(q, qshape, "q")
    ni, nj = scale_grid(rows, cols, block, transpose)
    if recip is None:
        recip = colmajor_empty(ni, nj, x.device)
    _check_scales(recip, (ni, nj), "recip")
    check(lib.fp8_blockwise_quant(x.data_ptr(), rows, cols, x.stride(0), BLOCKS[block],
                                  int(bool(transpose)), q.data_ptr(), q.stride(0),
                                  recip.data_ptr(), recip.stride(0), recip.stride(1), _stream(x)))
    return q, recip


@_on_tensor_device
def fp8_blockwise_quant_dual(x, block="1x128", q=None, recip=None, qt=None, recip_t=None,
                             stream_t=False):
    """Both layouts from one read of x: returns (q, recip, qt, recip_t), equal
    to fp8_blockwise_quant(x, block) and fp8_blockwise_quant(x, block,
    transpose=True).  stream_t writes qt with nontemporal stores (codes read
    only much later; the same bits)."""
    lib = load_library()
    _need_cuda(x)
    _rowmajor(x, "x")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if qt is None:
        qt = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
    _check_codes_out(q, (rows, cols), "q")
    _check_codes_out(qt, (cols, rows), "qt")
    ni, nj = scale_grid(rows, cols, block, False)
    ti, tj = scale_grid(rows, cols, block, True)
    if recip is None:
        recip = colmajor_empty(ni, nj, x.device)
    if recip_t is None:
        recip_t = colmajor_empty(ti, tj, x.device)
    _check_scales(recip, (ni, nj), "recip")
    _check_scales(recip_t, (ti, tj), "recip_t")
    check(lib.fp8_blockwise_quant_dual(x.data_ptr(), rows, cols, x.stride(0), BLOCKS[block],
                                       q.data_ptr(), q.stride(0), recip.data_ptr(), recip.stride(0),
                                       recip.stride(1), qt.data_ptr(), qt.stride(0),
                                       recip_t.data_ptr(), recip_t.stride(0), recip_t.stride(1),
                                       1 if stream_t else 0, _stream(x)))
    return q, recip, qt, recip_t


@_on_tensor_device
def fp8_tensorwise_quant(x, q=None, recip=None):
    """Per-tensor quantization: (q uint8 like x, recip fp32 [1] on device)."""
    lib = load_library()
    _need_cuda(x)
    _rowmajor(x, "x")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    _check_codes_out(q, (rows, cols), "q")
    if recip is None:
        recip = torch.empty(1, dtype=torch.float32, device=x.device)
    if recip.numel() != 1 or recip.dtype != torch.float32:
        raise ValueError("recip must be a one-element float32 tensor")
    nws = lib.fp8bw_tensorwise_quant_ws_bytes(rows, cols)
    ws = torch.empty(nws, dtype=torch.uint8, device=x.device)
    check(lib.fp8_tensorwise_quant(x.data_ptr(), rows, cols, x.stride(0), q.data_ptr(), q.stride(0),
                                   recip.data_ptr(), ws.data_ptr(), nws, _stream(x)))
    return q, recip


@_on_tensor_device
def fp8_tensorwise_quant_noalloc(x, q, recip):
    """fp8_tensorwise_quant with no workspace: the library keeps the partial
    amaxes in its own per-device array.  q (uint8 like x) and recip (fp32
    [1]) are the caller's; nothing is allocated here or in the library."""
    lib = load_library()
    _need_cuda(x)
    _rowmajor(x, "x")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    rows, cols = x.shape
    _check_codes_out(q, (rows, cols), "q")
    if recip.numel() != 1 or recip.dtype != torch.float32:
        raise ValueError("recip must be a one-element float32 tensor")
    check(lib.fp8_tensorwise_quant_noalloc(x.data_ptr(), rows, cols, x.stride(0), q.data_ptr(),
                                           q.stride(0), recip.data_ptr(), _stream(x)))
    return q, recip


def _check_bias(bias, N, device):
    if bias is None:
        return
    if bias.dtype != torch.bfloat16 or bias.dim() != 1 or bias.shape[0] != N or bias.stride(0) != 1:
        raise ValueError(f"bias must be a contiguous bf16 [{N}] tensor")
    if bias.device != device:
        raise ValueError("bias must be on the GEMM's device")


@_on_tensor_device
def fp8_scaled_gemm_blockwise(a, ra, b, rb, b_block="128x128", out_dtype=torch.bfloat16,
                              out=None, config=None, splits=None, bias=None):
    """out[M, N] = blockwise-scaled A . B^T (see include/fp8bw.h).

    a uint8 [M, K], ra fp32 [M, K/128] (column-major), b uint8 [N, K], rb fp32
    [N/128 or N, K/128].  config/splits force a tile configuration / split-K
    count (None = built-in choice)."""
    lib = load_library()
    _need_cuda(a, b, ra, rb)
    _rowmajor(a, "a")
    _rowmajor(b, "b")
    M, K = a.shape
    N = b.shape[0]
    _check_codes(a, b, K)
    kb = _cdiv(K, 128)
    if b_block not in BLOCKS:
        raise ValueError(f"b_block must be one of {sorted(BLOCKS)}")
    _check_scales(ra, (M, kb), "ra")
    _check_scales(rb, (N if b_block == "1x128" else _cdiv(N, 128), kb), "rb")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check_out(out, (M, N))
    args = (a.data_ptr(), a.stride(0), ra.data_ptr(), ra.stride(0), ra.stride(1),
            b.data_ptr(), b.stride(0), rb.data_ptr(), rb.stride(0), rb.stride(1),
            BLOCKS[b_block], M, N, K, out.data_ptr(), out.stride(0), OUT_DTYPES[out.dtype])
    _check_bias(bias, N, a.device)
    if bias is not None:
        if config is not None or splits is not None:
            raise ValueError("bias is not combined with a forced config/splits")
        nws = lib.fp8bw_gemm_blockwise_ws_bytes(M, N, K)
        ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=a.device)
        check(lib.fp8_scaled_gemm_blockwise_bias(*args[:14], bias.data_ptr(), *args[14:],
                                                 ws.data_ptr(), nws, _stream(a)))
        return out
    if config is None and splits is None:
        nws = lib.fp8bw_gemm_blockwise_ws_bytes(M, N, K)
        ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=a.device)
        check(lib.fp8_scaled_gemm_blockwise(*args, ws.data_ptr(), nws, _stream(a)))
    else:
        s = 0 if splits is None else int(splits)
        if s > 0:
            nws = lib.fp8bw_gemm_ws_bytes_for_split(M, N, s)
        else:
            nws = lib.fp8bw_gemm_blockwise_ws_bytes(M, N, K)
        ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=a.device)
        check(lib.fp8_scaled_gemm_blockwise_cfg(*args, -1 if config is None else int(config), s,
                                                ws.data_ptr(), nws, _stream(a)))
    return out


@_on_tensor_device
def fp8_scaled_gemm_blockwise_kn(a, ra, b_kn, rb, b_block="128x128", out_dtype=torch.bfloat16,
                                 out=None):
    """out[M, N] = blockwise-scaled A . B with B given in [K, N] layout
    (N contiguous), e.g. a weight's codes W [N_w, K_w] used as the B of
    dX = dY . W without a transposed copy (see include/fp8bw.h).

    a uint8 [M, K], ra fp32 [M, K/128], b_kn uint8 [K, N], rb fp32
    [N/128 or N, K/128] indexed by (output column block, K block)."""
    lib = load_library()
    _need_cuda(a, b_kn, ra, rb)
    _rowmajor(a, "a")
    _rowmajor(b_kn, "b_kn")
    M, K = a.shape
    if b_kn.dim() != 2 or b_kn.shape[0] != K:
        raise ValueError(f"b_kn must be [K={K}, N]")
    N = b_kn.shape[1]
    _check_codes(a, b_kn.t(), K)
    kb = _cdiv(K, 128)
    if b_block not in BLOCKS:
        raise ValueError(f"b_block must be one of {sorted(BLOCKS)}")
    _check_scales(ra, (M, kb), "ra")
    _check_scales(rb, (N if b_block == "1x128" else _cdiv(N, 128), kb), "rb")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check_out(out, (M, N))
    nws = lib.fp8bw_gemm_blockwise_ws_bytes(M, N, K)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=a.device)
    check(lib.fp8_scaled_gemm_blockwise_kn(
        a.data_ptr(), a.stride(0), ra.data_ptr(), ra.stride(0), ra.stride(1), b_kn.data_ptr(),
        b_kn.stride(0), rb.data_ptr(), rb.stride(0), rb.stride(1), BLOCKS[b_block], M, N, K,
        out.data_ptr(), out.stride(0), OUT_DTYPES[out.dtype], ws.data_ptr(), nws, _stream(a)))
    return out


def fp8bw_gemm_num_configs():
    return load_library().fp8bw_gemm_num_configs()


def gemm_plan(M, N, K, b_block="128x128"):
    """How the library runs an M x N x K blockwise GEMM (contiguous operands,
    column-major scales) on the current device: tile configuration,
    whole-problem split count, leftover-tile split count, tiles, tiles run
    unsplit and workspace bytes."""
    import ctypes
    info = (ctypes.c_int64 * 6)()
    check(load_library().fp8bw_gemm_blockwise_plan(M, N, K, BLOCKS[b_block], info))
    keys = ("config", "splits", "tail_splits", "tiles", "tiles_full", "ws_bytes")
    return dict(zip(keys, (int(v) for v in info)))


@_on_tensor_device
def fp8_scaled_gemm_tensorwise(a, ra, b, rb, out_dtype=torch.bfloat16, out=None, bias=None):
    """out[M, N] = (A . B^T) * ra * rb with one-element device scales."""
    lib = load_library()
    _need_cuda(a, b, ra, rb)
    _rowmajor(a, "a")
    _rowmajor(b, "b")
    M, K = a.shape
    N = b.shape[0]
    _check_codes(a, b, K)
    if ra.numel() != 1 or rb.numel() != 1:
        raise ValueError("tensorwise scales are one-element tensors")
    if ra.dtype != torch.float32 or rb.dtype != torch.float32:
        raise ValueError("tensorwise scales are float32")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check_out(out, (M, N))
    _check_bias(bias, N, a.device)
    if bias is not None:
        check(lib.fp8_scaled_gemm_tensorwise_bias(a.data_ptr(), a.stride(0), ra.data_ptr(),
                                                  b.data_ptr(), b.stride(0), rb.data_ptr(), M, N, K,
                                                  bias.data_ptr(), out.data_ptr(), out.stride(0),
                                                  OUT_DTYPES[out.dtype], _stream(a)))
        return out
    check(lib.fp8_scaled_gemm_tensorwise(a.data_ptr(), a.stride(0), ra.data_ptr(), b.data_ptr(),
                                         b.stride(0), rb.data_ptr(), M, N, K, out.data_ptr(),
                                         out.stride(0), OUT_DTYPES[out.dtype], _stream(a)))
    return out


@_on_tensor_device
def fp8_scaled_grouped_gemm_blockwise(a, ra, b, rb, group_end, out_dtype=torch.bfloat16, out=None):
    """Grouped blockwise GEMM: rows [group_end[g-1], group_end[g]) of a
    (uint8 [M, K], ra fp32 [M, K/128] column-major) times b[g]^T (uint8
    [G, N, K], rb fp32 [G, N/128, K/128], any strides) -> out [M, N].
    group_end: device int32 [G], cumulative."""
    lib = load_library()
    _need_cuda(a, b, ra, rb, group_end)
    _rowmajor(a, "a")
    M, K = a.shape
    if b.dim() != 3 or b.shape[2] != K or b.stride(2) != 1:
        raise ValueError("b must be uint8 [G, N, K] with contiguous rows")
    G, N = b.shape[0], b.shape[1]
    if a.dtype != torch.uint8 or b.dtype != torch.uint8:
        raise ValueError("codes are uint8 tensors")
    kb = _cdiv(K, 128)
    _check_scales(ra, (M, kb), "ra")
    if ra.stride(0) != 1 and M > 1:
        raise ValueError("ra of the grouped GEMM must be column-major (unit row stride)")
    _check_scales(rb, (G, _cdiv(N, 128), kb), "rb")
    if group_end.dtype != torch.int32 or group_end.shape != (G,) or group_end.stride(0) != 1:
        raise ValueError("group_end must be a contiguous int32 [G] tensor")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check_out(out, (M, N))
    check(lib.fp8_scaled_grouped_gemm_blockwise(
        a.data_ptr(), a.stride(0), ra.data_ptr(), ra.stride(1), b.data_ptr(), b.stride(1),
        b.stride(0), rb.data_ptr(), rb.stride(1), rb.stride(2), rb.stride(0), G,
        group_end.data_ptr(), M, N, K, out.data_ptr(), out.stride(0), OUT_DTYPES[out.dtype],
        _stream(a)))
    return out


def linear_saved_bytes(M, N, K):
    """Bytes of the buffer fp8_linear_fwd_save fills for fp8_linear_bwd."""
    return load_library().fp8bw_linear_saved_bytes(M, N, K)


def linear_workspace(M, N, K, which, device):
    n = load_library().fp8bw_linear_ws_bytes(M, N, K, which)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _linear(name, which, p0, p1, out_shape, M, N, K, ws):
    lib = load_library()
    _need_cuda(p0, p1)
    if not (p0.is_contiguous() and p1.is_contiguous()):
        raise ValueError("linear inputs must be contiguous")
    out = torch.empty(out_shape, dtype=torch.bfloat16, device=p0.device)
    if ws is None:
        ws = linear_workspace(M, N, K, which, p0.device)
    check(getattr(lib, name)(p0.data_ptr(), p1.data_ptr(), out.data_ptr(), M, N, K,
                             ws.data_ptr(), ws.numel(), _stream(p0)))
    return out


def _bf16_2d(*ts):
    for t in ts:
        if t.dim() != 2 or t.dtype != torch.bfloat16:
            raise ValueError("linear inputs are 2-D bf16 tensors")


@_on_tensor_device
def fp8_linear_fwd(x, w, ws=None):
    """Y[M, N] = X . W^T (X 1x128, W 128x128), bf16."""
    _bf16_2d(x, w)
    M, K = x.shape
    N = w.shape[0]
    _check_shape(w, (N, K), "w")
    return _linear("fp8_linear_fwd", 0, x, w, (M, N), M, N, K, ws)


@_on_tensor_device
def fp8_linear_dgrad(dy, w, ws=None):
    """dX[M, K] = dY . W (dY 1x128, W^T 128x128), bf16."""
    _bf16_2d(dy, w)
    M, N = dy.shape
    K = w.shape[1]
    _check_shape(w, (N, K), "w")
    return _linear("fp8_linear_dgrad", 1, dy, w, (M, K), M, N, K, ws)


@_on_tensor_device
def fp8_linear_fwd_save(x, w, ws=None):
    """Y[M, N] = X . W^T with fused quantization: returns (Y, saved), where
    saved (uint8, device) holds the X^T codes and scales that fp8_linear_bwd
    needs (see include/fp8bw.h)."""
    _bf16_2d(x, w)
    M, K = x.shape
    N = w.shape[0]
    _check_shape(w, (N, K), "w")
    lib = load_library()
    _need_cuda(x, w)
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("linear inputs must be contiguous")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    saved = torch.empty(max(linear_saved_bytes(M, N, K), 1), dtype=torch.uint8, device=x.device)
    if ws is None:
        ws = linear_workspace(M, N, K, 3, x.device)
    check(lib.fp8_linear_fwd_save(x.data_ptr(), w.data_ptr(), y.data_ptr(), M, N, K,
                                  saved.data_ptr(), saved.numel(), ws.data_ptr(), ws.numel(),
                                  _stream(x)))
    return y, saved


@_on_tensor_device
def fp8_linear_bwd(dy, w, saved, need_dx=True, need_dw=True, ws=None):
    """(dX[M, K], dW[N, K]) from dY[M, N], the forward's bf16 W[N, K] and
    the saved buffer of fp8_linear_fwd_save (dY quantized once, W^T right
    before the dgrad GEMM); a gradient not needed is None."""
    _bf16_2d(dy, w)
    M, N = dy.shape
    K = w.shape[1]
    _check_shape(w, (N, K), "w")
    lib = load_library()
    _need_cuda(dy, w, saved)
    if not (dy.is_contiguous() and w.is_contiguous()):
        raise ValueError("dy and w must be contiguous")
    if saved.dtype != torch.uint8 or saved.dim() != 1:
        raise ValueError("saved must be the 1-D uint8 buffer from fp8_linear_fwd_save")
    dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device) if need_dx else None
    dw = torch.empty((N, K), dtype=torch.bfloat16, device=dy.device) if need_dw else None
    if ws is None:
        ws = linear_workspace(M, N, K, 4, dy.device)
    check(lib.fp8_linear_bwd(dy.data_ptr(), w.data_ptr(), saved.data_ptr(), saved.numel(),
                             dx.data_ptr() if dx is not None else None,
                             dw.data_ptr() if dw is not None else None, M, N, K, ws.data_ptr(),
                             ws.numel(), _stream(dy)))
    return dx, dw


@_on_tensor_device
def fp8_linear_wgrad(dy, x, ws=None):
    """dW[N, K] = dY^T . X (1x128 x 1x128 along M), bf16."""
    _bf16_2d(dy, x)
    M, N = dy.shape
    K = x.shape[1]
    _check_shape(x, (M, K), "x")
    return _linear("fp8_linear_wgrad", 2, dy, x, (N, K), M, N, K, ws)


# ---------------------------------------------------------------------------
# The operators around the linear in a training step (include/fp8bw.h):
# RMS norm, vocabulary cross entropy, AdamW.

class RMSNormOut(NamedTuple):
    """Outputs of rms_norm_fwd; what was not asked for is None."""
    s: torch.Tensor                  # x + residual in bf16 (x itself without a residual)
    rstd: torch.Tensor               # fp32 [rows]
    y: Optional[torch.Tensor]        # bf16 [rows, cols]
    q: Optional[torch.Tensor]        # uint8 codes [rows, cols]
    recip: Optional[torch.Tensor]    # fp32 [rows, ceil(cols / 128)], column-major
    qt: Optional[torch.Tensor]       # uint8 codes [cols, rows]
    recip_t: Optional[torch.Tensor]  # fp32 [cols, ceil(rows / 128)], column-major


def _bf16_matrix(t, name, shape=None):
    _rowmajor(t, name)
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bf16")
    if shape is not None:
        _check_shape(t, shape, name)


def _norm_weight(weight, cols):
    if weight.dim() != 1 or weight.dtype not in OUT_DTYPES or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous bf16 or float32 vector")
    _check_shape(weight, (cols,), "weight")


def _vector(t, n, dtype, name):
    if t.dtype != dtype or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector")
    _check_shape(t, (n,), name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ld(t):
    return 0 if t is None else t.stride(0)


@_on_tensor_device
def rms_norm_fwd(x, weight, residual=None, eps=1e-6, y=True, q=False, qt=False, s=None):
    """RMS norm of s = x + residual (bf16) times weight, as RMSNormOut.

    x, residual bf16 [rows, cols] (unit column stride); weight bf16 or fp32
    [cols].  y, q, qt choose the outputs: bf16, E4M3 codes in 1x128 blocks
    along the columns, and transposed codes in 1x128 blocks along the rows
    (rows % 16 == 0).  s: where to write x + residual, possibly x or residual
    itself (default: a new tensor)."""
    lib = load_library()
    _need_cuda(x, weight)
    _bf16_matrix(x, "x")
    rows, cols = x.shape
    _norm_weight(weight, cols)
    dev = x.device
    given = s
    if residual is not None:
        _bf16_matrix(residual, "residual", (rows, cols))
        if s is None:
            s = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
        _bf16_matrix(s, "s", (rows, cols))
    elif s is not None:
        raise ValueError("s is written only with a residual")
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    ty = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev) if y else None
    tq = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if q else None
    # column-major scales in one allocation call (no view to build)
    tr = torch.empty_strided((rows, _cdiv(cols, 128)), (1, max(rows, 1)), dtype=torch.float32,
                             device=dev) if q else None
    tqt = torch.empty((cols, rows), dtype=torch.uint8, device=dev) if qt else None
    trt = torch.empty_strided((cols, _cdiv(rows, 128)), (1, max(cols, 1)), dtype=torch.float32,
                              device=dev) if qt else None
    check(lib.fp8bw_rms_norm_fwd(
        x.data_ptr(), x.stride(0), _ptr(residual), _ld(residual), weight.data_ptr(),
        OUT_DTYPES[weight.dtype], float(eps), rows, cols, _ptr(s), _ld(s), rstd.data_ptr(),
        _ptr(ty), _ld(ty), _ptr(tq), _ld(tq), _ptr(tr), tr.stride(0) if q else 0,
        tr.stride(1) if q else 0, _ptr(tqt), _ld(tqt), _ptr(trt), trt.stride(0) if qt else 0,
        trt.stride(1) if qt else 0, _stream(x)))
    if given is not None:
        torch.autograd.graph.increment_version(given)
    return RMSNormOut(x if residual is None else s, rstd, ty, tq, tr, tqt, trt)


@_on_tensor_device
def rms_norm_bwd(dy, s, rstd, weight, dres=None):
    """(dx, dweight) of rms_norm_fwd from dy, its s and rstd, and dres, the
    gradient that reaches s past the norm (or None).  dx bf16 is the gradient
    of x and of the residual; dweight has the weight's type."""
    lib = load_library()
    _need_cuda(dy, s, rstd, weight)
    _bf16_matrix(dy, "dy")
    rows, cols = dy.shape
    _bf16_matrix(s, "s", (rows, cols))
    _vector(rstd, rows, torch.float32, "rstd")
    _norm_weight(weight, cols)
    if dres is not None:
        _bf16_matrix(dres, "dres", (rows, cols))
    dx = torch.empty((rows, cols), dtype=torch.bfloat16, device=dy.device)
    if rows == 0:
        return dx, torch.zeros_like(weight)
    dweight = torch.empty_like(weight)
    nws = lib.fp8bw_rms_norm_bwd_ws_bytes(rows, cols)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=dy.device)
    check(lib.fp8bw_rms_norm_bwd(dy.data_ptr(), dy.stride(0), s.data_ptr(), s.stride(0),
                                 rstd.data_ptr(), weight.data_ptr(), OUT_DTYPES[weight.dtype],
                                 _ptr(dres), _ld(dres), rows, cols, dx.data_ptr(), dx.stride(0),
                                 dweight.data_ptr(), ws.data_ptr(), nws, _stream(dy)))
    return dx, dweight


def _check_xent(h, w, target):
    _need_cuda(h, w, target)
    _bf16_matrix(h, "h")
    T, K = h.shape
    _bf16_matrix(w, "w")
    _check_shape(w, (w.shape[0], K), "w")
    _vector(target, T, torch.int64, "target")
    return T, w.shape[0], K


@_on_tensor_device
def linear_xent_fwd(h, w, target, ignore_index=-100):
    """(loss, lse), both fp32 [T], of softmax cross entropy with logits
    h . w^T: h bf16 [T, K], w bf16 [V, K], target int64 [T].  A token whose
    target is ignore_index has loss 0; any other target outside the
    vocabulary gives NaN."""
    lib = load_library()
    T, V, K = _check_xent(h, w, target)
    loss = torch.empty(T, dtype=torch.float32, device=h.device)
    lse = torch.empty(T, dtype=torch.float32, device=h.device)
    nws = lib.fp8bw_linear_xent_ws_bytes(T, V, K, 0)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=h.device)
    check(lib.fp8bw_linear_xent_fwd(h.data_ptr(), h.stride(0), w.data_ptr(), w.stride(0),
                                    target.data_ptr(), int(ignore_index), T, V, K, loss.data_ptr(),
                                    lse.data_ptr(), ws.data_ptr(), nws, _stream(h)))
    return loss, lse


@_on_tensor_device
def linear_xent_bwd(dloss, h, w, target, lse, ignore_index=-100, need_dh=True, need_dw=True,
                    loss=None):
    """(dh, dw), bf16, of linear_xent_fwd from dloss fp32 [T], one weight per
    token's loss, and the forward's lse; a gradient not needed is None.

    loss: the forward's losses, from which the target's entry of the softmax's
    gradient, p - 1, comes to fp32's relative precision; without them it is off
    by the rounding of lse, which is all of it for very confident tokens."""
    lib = load_library()
    T, V, K = _check_xent(h, w, target)
    _need_cuda(dloss, lse)
    _vector(dloss, T, torch.float32, "dloss")
    _vector(lse, T, torch.float32, "lse")
    if loss is not None:
        _vector(loss, T, torch.float32, "loss")
    dh = torch.empty((T, K), dtype=torch.bfloat16, device=h.device) if need_dh else None
    dw = torch.empty((V, K), dtype=torch.bfloat16, device=h.device) if need_dw else None
    nws = lib.fp8bw_linear_xent_ws_bytes(T, V, K, 1)
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=h.device)
    check(lib.fp8bw_linear_xent_bwd_loss(dloss.data_ptr(), h.data_ptr(), h.stride(0), w.data_ptr(),
                                         w.stride(0), target.data_ptr(), int(ignore_index),
                                         lse.data_ptr(), _ptr(loss), T, V, K, _ptr(dh), _ld(dh),
                                         _ptr(dw), _ld(dw), ws.data_ptr(), nws, _stream(h)))
    return dh, dw


def adamw_scales(n):
    """Scales of n elements of 8-bit AdamW state."""
    return _cdiv(n, 128)


def _adamw_list(ts, n, name):
    if len(ts) != n:
        raise ValueError(f"{len(ts)} {name} for {n} params")
    return ts


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, *, step, lr, beta1=0.9, beta2=0.999, eps=1e-8,
               weight_decay=0.0, exp_avg_scales=None, root_scales=None, masters=None,
               grad_scale=None, seed=None, ordinals=None):
    """One AdamW step over lists of contiguous tensors, in place.

    params and grads bf16 or fp32.  With fp32 exp_avgs and exp_avg_sqs the
    states are the moments; with uint8 (or float8_e4m3fn) ones they are E4M3
    codes of m and of sqrt(v), whose scales per 128 elements (adamw_scales)
    are exp_avg_scales and root_scales.  masters: fp32 weights behind bf16
    params (a list, None for tensors without one).  grad_scale: one-element
    fp32 tensor that multiplies every gradient.  seed: a new integer each step
    to round codes and bf16 params at random; None rounds to nearest.  ordinals:
    one distinct number below 2^20 per tensor, which with the seed picks its
    random numbers; default its place in the lists.  Calls that share a seed (one
    per parameter group) give every tensor another."""
    lib = load_library()
    n = len(params)
    if n == 0:
        return
    eight = exp_avgs[0].dtype in CODE_DTYPES if len(exp_avgs) else False
    if eight != (exp_avg_scales is not None) or eight != (root_scales is not None):
        raise ValueError("exp_avg_scales and root_scales belong to 8-bit states")
    for ts, name in ((grads, "grads"), (exp_avgs, "exp_avgs"), (exp_avg_sqs, "exp_avg_sqs"),
                     (exp_avg_scales, "exp_avg_scales"), (root_scales, "root_scales"),
                     (masters, "masters")):
        if ts is not None:
            _adamw_list(ts, n, name)
    # Checks and addresses list by list, one attribute at a time, and the C
    # array's words in one go: about 1 us a tensor, a small model's whole cost.
    device = params[0].device
    index = device.index if device.type == "cuda" else -1
    numels = [t.numel() for t in params]
    state_dtypes = CODE_DTYPES if eight else (torch.float32,)
    here, yes = {index}, {True}
    kinds = []
    for ts, dtypes, name in ((params, OUT_DTYPES, "params"), (grads, OUT_DTYPES, "grads"),
                             (exp_avgs, state_dtypes, "exp_avgs"),
                             (exp_avg_sqs, state_dtypes, "exp_avg_sqs")):
        if index < 0 or {t.get_device() for t in ts} != here:
            raise ValueError("fp8bw ops take CUDA (HIP) tensors on one device")
        if [t.numel() for t in ts] != numels or {t.is_contiguous() for t in ts} != yes:
            raise ValueError("params, grads and states must be contiguous and of equal size")
        kinds.append({t.dtype for t in ts})
        if not kinds[-1] <= set(dtypes):
            raise ValueError(f"{name} must be of {' or '.join(str(d) for d in dtypes)}")
    zeros = [0] * n
    blocks = [(_cdiv(m, 128),) for m in numels] if eight else None
    scales = []
    for ts in (exp_avg_scales, root_scales):
        if ts is None:
            scales.append(zeros)
            continue
        if {t.get_device() for t in ts} != here:
            raise ValueError("fp8bw ops take CUDA (HIP) tensors on one device")
        if ([t.shape for t in ts] != blocks or {t.dtype for t in ts} != {torch.float32}
                or {t.is_contiguous() for t in ts} != yes):
            raise ValueError("scales must be contiguous float32 vectors, one element per 128 of the state")
        scales.append([t.data_ptr() for t in ts])
    if masters is None:
        master_ptrs = zeros
    else:
        for t, m in zip(masters, numels):
            if t is not None and (t.get_device() != index or t.dtype != torch.float32
                                  or not t.is_contiguous() or t.numel() != m):
                raise ValueError("masters must be contiguous float32 tensors like params")
        master_ptrs = [0 if t is None else t.data_ptr() for t in masters]
    # AdamwTensor's fields in order, its two int types in one word
    if len(kinds[0]) == len(kinds[1]) == 1:
        types = [OUT_DTYPES[params[0].dtype] | OUT_DTYPES[grads[0].dtype] << 32] * n
    else:
        types = [OUT_DTYPES[p.dtype] | OUT_DTYPES[g.dtype] << 32 for p, g in zip(params, grads)]
    places = range(n) if ordinals is None else [int(o) for o in ordinals]
    if ordinals is not None and (len(places) != n or len(set(places)) != n or min(places) < 0
                                 or max(places) >= 1 << 20):
        raise ValueError("ordinals must be distinct numbers below 2^20, one per param")
    fields = ([t.data_ptr() for t in params], [t.data_ptr() for t in grads],
              [t.data_ptr() for t in exp_avgs], [t.data_ptr() for t in exp_avg_sqs],
              *scales, master_ptrs, numels, types)
    # a tensor's ordinal is its place in the array; the places between stay empty
    count = n if ordinals is None else max(places) + 1
    words = [0] * (9 * count)
    if ordinals is None:
        for k, column in enumerate(fields):
            words[k::9] = column
    else:
        for place, row in zip(places, zip(*fields)):
            words[9 * place:9 * place + 9] = row
    arr = (AdamwTensor * count).from_buffer(array.array("q", words))
    if grad_scale is not None and (grad_scale.device != device or grad_scale.dtype != torch.float32
                                   or grad_scale.numel() != 1):
        raise ValueError("grad_scale must be a one-element float32 tensor on the params' device")
    args = (arr, count, int(eight), int(step), float(lr), float(beta1), float(beta2), float(eps),
            float(weight_decay), _ptr(grad_scale), int(seed is not None),
            0 if seed is None else int(seed) & 0xFFFFFFFFFFFFFFFF, _stream(params[0]))
    if index == torch._C._cuda_getDevice():
        check(lib.fp8bw_adamw_step(*args))
    else:
        with torch.cuda.device(device):
            check(lib.fp8bw_adamw_step(*args))
    # a graph that saved a parameter refuses to run backward through the new values
    torch.autograd.graph.increment_version(params)


# ---------------------------------------------------------------------------
# The operators around the grouped GEMM in a mixture-of-experts layer
# (include/fp8bw.h): sort, gather, combine, gated activation, weight gradients.

class MoeTable(NamedTuple):
    """Slots (token, choice) sorted by expert, as moe_sort makes it."""
    row: torch.Tensor         # int32 [tokens, topk]: a slot's row, -1 without an expert
    source: torch.Tensor      # int32 [rows]: a row's slot t * topk + j, -1 without one
    group_end: torch.Tensor   # int32 [experts], cumulative: the grouped GEMM's table


class Rows(NamedTuple):
    """Layouts of a [rows, cols] result; what was not asked for is None."""
    y: Optional[torch.Tensor]        # bf16 [rows, cols]
    q: Optional[torch.Tensor]        # uint8 codes [rows, cols]
    recip: Optional[torch.Tensor]    # fp32 [rows, blocks], column-major
    qt: Optional[torch.Tensor]       # uint8 codes [cols, rows]
    recip_t: Optional[torch.Tensor]  # fp32 [cols, ceil(rows / 128)], column-major


class SwigluOut(NamedTuple):
    """Outputs of swiglu_fwd; what was not asked for is None."""
    y: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    recip: Optional[torch.Tensor]
    qt: Optional[torch.Tensor]
    recip_t: Optional[torch.Tensor]
    hq: Optional[torch.Tensor]       # uint8 codes [rows, 2 ffn] of h
    h_recip: Optional[torch.Tensor]  # fp32 [rows, 2 ceil(ffn / 128)], column-major


class SwigluGrads(NamedTuple):
    """Outputs of swiglu_bwd; what was not asked for is None."""
    dh: Optional[torch.Tensor]           # bf16 [rows, 2 ffn]
    q: Optional[torch.Tensor]            # uint8 codes [rows, 2 ffn] of dh
    recip: Optional[torch.Tensor]        # fp32 [rows, 2 ceil(ffn / 128)], column-major
    qt: Optional[torch.Tensor]           # uint8 codes [2 ffn, rows] of dh^T
    recip_t: Optional[torch.Tensor]      # fp32 [2 ffn, ceil(rows / 128)], column-major
    act_qt: Optional[torch.Tensor]       # uint8 codes [ffn, rows] of the activation's transpose
    act_recip_t: Optional[torch.Tensor]  # fp32 [ffn, ceil(rows / 128)], column-major


def _matrix_empty(rows, cols, dtype, device):
    # empty_strided costs 1.4 us, torch.empty 1.75: of a decoding step's calls, each
    # about 10 us on the host, that is what can be spared
    return torch.empty_strided((rows, cols), (max(cols, 1), 1), dtype=dtype, device=device)


def _codes_empty(rows, cols, blocks, device):
    """(codes [rows, cols], column-major scales [rows, blocks])."""
    return (_matrix_empty(rows, cols, torch.uint8, device),
            torch.empty_strided((rows, blocks), (1, max(rows, 1)), dtype=torch.float32, device=device))


def _layouts_empty(rows, cols, blocks, y, q, qt, device):
    """(Rows, the C struct that names its tensors)."""
    ty = tq = tr = tqt = trt = None
    if y:
        ty = _matrix_empty(rows, cols, torch.bfloat16, device)
    if q:
        tq, tr = _codes_empty(rows, cols, blocks, device)
    if qt:
        tqt, trt = _codes_empty(cols, rows, _cdiv(rows, 128), device)
    return (Rows(ty, tq, tr, tqt, trt),
            Layouts(_ptr(ty), cols, _ptr(tq), cols, _ptr(tr), 1, rows, _ptr(tqt), rows, _ptr(trt), 1, cols))


def _moe_table(table, device):
    """(tokens, topk, rows) of a table on `device`."""
    row, source, group_end = table
    index = device.index
    for t, dim, name in ((row, 2, "row"), (source, 1, "source"), (group_end, 1, "group_end")):
        if t.dtype != torch.int32 or t.dim() != dim or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"the table's {name} must be a contiguous int32 tensor of {dim} dimension"
                             f"{'s' if dim > 1 else ''} on {device}")
    return row.shape[0], row.shape[1], source.shape[0]


def _moe_weight(weight, tokens, topk):
    if weight.dtype not in OUT_DTYPES or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous bf16 or float32 tensor")
    _check_shape(weight, (tokens, topk), "weight")


def moe_rows(tokens, topk, experts, align=128):
    """Rows of moe_sort's table: what holds the slots however they fall."""
    return load_library().fp8bw_moe_rows(tokens, topk, experts, align)


@_on_tensor_device
def moe_sort(expert, experts, align=128):
    """MoeTable of slots sorted by expert, each expert's rows padded to a
    multiple of `align`.

    expert int32 or int64 [tokens, topk]; a number outside [0, experts) is no
    expert.  Slots of one expert keep their order."""
    lib = load_library()
    _need_cuda(expert)
    if expert.dim() != 2 or expert.dtype not in (torch.int32, torch.int64) or not expert.is_contiguous():
        raise ValueError("expert must be a contiguous int32 or int64 tensor [tokens, topk]")
    tokens, topk = expert.shape
    experts, align = int(experts), int(align)
    rows = lib.fp8bw_moe_rows(tokens, topk, experts, align)
    dev = expert.device
    row = _matrix_empty(tokens, topk, torch.int32, dev)
    source = torch.empty_strided((rows,), (1,), dtype=torch.int32, device=dev)
    group_end = torch.empty_strided((max(experts, 0),), (1,), dtype=torch.int32, device=dev)
    nws = lib.fp8bw_moe_sort_ws_bytes(tokens, topk, experts)
    ws = torch.empty(nws, dtype=torch.uint8, device=dev) if nws else None
    check(lib.fp8bw_moe_sort(expert.data_ptr(), 32 if expert.dtype == torch.int32 else 64, tokens, topk,
                             experts, align, rows, row.data_ptr(), source.data_ptr(),
                             group_end.data_ptr(), _ptr(ws), nws, _stream(expert)))
    return MoeTable(row, source, group_end)


@_on_tensor_device
def moe_gather(x, table, y=True, q=False, qt=False):
    """Rows of x bf16 [tokens, cols] in the table's order (zeros in rows without
    a slot): bf16, E4M3 codes in 1x128 blocks along the columns, and codes of
    the transpose in 1x128 blocks along the rows.  The gradient of y is
    moe_combine(dy, table)."""
    lib = load_library()
    _need_cuda(x)
    _bf16_matrix(x, "x")
    dev = x.device
    tokens, topk, rows = _moe_table(table, dev)
    cols = x.shape[1]
    if x.shape[0] != tokens:
        _check_shape(x, (tokens, cols), "x")
    out, c = _layouts_empty(rows, cols, _cdiv(cols, 128), y, q, qt, dev)
    check(lib.fp8bw_moe_gather(x.data_ptr(), x.stride(0), tokens, topk, table.row.data_ptr(),
                               table.source.data_ptr(), rows, cols, c, _stream(x)))
    return out


@_on_tensor_device
def moe_combine(y, table, weight=None):
    """bf16 [tokens, cols]: every token's rows of y bf16 [rows, cols] summed in
    fp32, times weight (fp32 or bf16 [tokens, topk]) if given."""
    lib = load_library()
    _need_cuda(y)
    _bf16_matrix(y, "y")
    tokens, topk, rows = _moe_table(table, y.device)
    cols = y.shape[1]
    _check_shape(y, (rows, cols), "y")
    if weight is not None:
        _moe_weight(weight, tokens, topk)
    out = _matrix_empty(tokens, cols, torch.bfloat16, y.device)
    check(lib.fp8bw_moe_combine(y.data_ptr(), y.stride(0), _ptr(weight),
                                1 if weight is None else OUT_DTYPES[weight.dtype], tokens, topk,
                                table.row.data_ptr(), rows, cols, out.data_ptr(), out.stride(0), _stream(y)))
    return out


@_on_tensor_device
def moe_combine_bwd(dout, y, table, weight, dy=True, q=False, qt=False, need_dweight=True):
    """(Rows, dweight) of moe_combine from dout bf16 [tokens, cols]: the
    gradient of its y in the layouts asked for (as moe_gather), and that of
    weight, in its type (None without need_dweight; y may then be None)."""
    lib = load_library()
    _need_cuda(dout, weight)
    _bf16_matrix(dout, "dout")
    tokens, topk, rows = _moe_table(table, dout.device)
    cols = dout.shape[1]
    _check_shape(dout, (tokens, cols), "dout")
    _moe_weight(weight, tokens, topk)
    dweight = None
    if need_dweight:
        _need_cuda(y)
        _bf16_matrix(y, "y", (rows, cols))
        dweight = torch.empty_like(weight)
        if cols == 0:
            dweight.zero_()
    out, c = _layouts_empty(rows, cols, _cdiv(cols, 128), dy, q, qt, dout.device)
    if cols:
        check(lib.fp8bw_moe_combine_bwd(dout.data_ptr(), dout.stride(0), y.data_ptr() if need_dweight else None,
                                        y.stride(0) if need_dweight else 0, weight.data_ptr(),
                                        OUT_DTYPES[weight.dtype], tokens, topk, table.row.data_ptr(),
                                        table.source.data_ptr(), rows, cols, c, _ptr(dweight), _stream(dout)))
    return out, dweight


def _halves(t, name):
    if t.shape[1] % 2:
        raise ValueError(f"{name} must have an even number of columns")
    return t.shape[1] // 2


@_on_tensor_device
def swiglu_fwd(h, y=True, q=False, qt=False, save=False):
    """SwigluOut of v = silu(gate) * up, h = [gate | up] bf16 [rows, 2 ffn].

    y, q, qt choose v's layouts (as moe_gather).  save: also h itself in E4M3
    codes with a scale per 1x128 block of each half, which swiglu_bwd takes in
    the place of h at half its bytes."""
    lib = load_library()
    _need_cuda(h)
    _bf16_matrix(h, "h")
    rows, ffn = h.shape[0], _halves(h, "h")
    out, c = _layouts_empty(rows, ffn, _cdiv(ffn, 128), y, q, qt, h.device)
    hq = hr = None
    if save:
        hq, hr = _codes_empty(rows, 2 * ffn, 2 * _cdiv(ffn, 128), h.device)
    check(lib.fp8bw_swiglu_fwd(h.data_ptr(), h.stride(0), rows, ffn, c, _ptr(hq), 2 * ffn, _ptr(hr), 1, rows,
                               _stream(h)))
    return SwigluOut(*out, hq, hr)


@_on_tensor_device
def swiglu_bwd(dy, h, h_recip=None, dh=True, q=False, qt=False, act_qt=False):
    """SwigluGrads of swiglu_fwd from dy bf16 [rows, ffn] and h: bf16, or the
    codes of a checkpoint with its scales h_recip.

    dh, q, qt choose the layouts of the gradient of h (q in 1x128 blocks of each
    half); act_qt makes the activation's transposed codes again, the operand of
    the weight gradient of the product behind it.  For act_qt alone dy is not
    read and may be None."""
    lib = load_library()
    if dy is None and not (dh or q or qt):
        _need_cuda(h)
        if h.dim() != 2:
            raise ValueError("h must be a 2-D tensor")
        rows, ffn = h.shape[0], _halves(h, "h")
    else:
        _need_cuda(dy, h)
        _bf16_matrix(dy, "dy")
        rows, ffn = dy.shape
    if h_recip is None:
        _bf16_matrix(h, "h", (rows, 2 * ffn))
    else:
        _check_codes_out(h, (rows, 2 * ffn), "h")
        _check_scales(h_recip, (rows, 2 * _cdiv(ffn, 128)), "h_recip")
    out, c = _layouts_empty(rows, 2 * ffn, 2 * _cdiv(ffn, 128), dh, q, qt, h.device)
    tq = tr = None
    if act_qt:
        tq, tr = _codes_empty(ffn, rows, _cdiv(rows, 128), h.device)
    check(lib.fp8bw_swiglu_bwd(_ptr(dy), 0 if dy is None else dy.stride(0), h.data_ptr(), h.stride(0), _ptr(h_recip),
                               0 if h_recip is None else h_recip.stride(0),
                               0 if h_recip is None else h_recip.stride(1), rows, ffn, c, _ptr(tq), rows,
                               _ptr(tr), 1, ffn, _stream(h)))
    return SwigluGrads(*out, tq, tr)


@_on_tensor_device
def fp8_scaled_grouped_gemm_blockwise_wgrad(a, ra, b, rb, group_end, out_dtype=torch.bfloat16, out=None):
    """Weight gradients of a grouped GEMM: out[g] = A . B^T over the columns
    [group_end[g-1], group_end[g]) of a uint8 [M, K] and b uint8 [N, K], the
    transposed codes of dY and X in 1x128 blocks with scales ra fp32 [M, K/128]
    and rb fp32 [N, K/128] -> out [G, M, N].  group_end: device int32 [G],
    cumulative multiples of 128 (moe_sort with align 128)."""
    lib = load_library()
    _need_cuda(a, b, ra, rb, group_end)
    _rowmajor(a, "a")
    _rowmajor(b, "b")
    M, K = a.shape
    N = b.shape[0]
    _check_codes(a, b, K)
    kb = _cdiv(K, 128)
    _check_scales(ra, (M, kb), "ra")
    _check_scales(rb, (N, kb), "rb")
    if group_end.dtype != torch.int32 or group_end.dim() != 1 or not group_end.is_contiguous():
        raise ValueError("group_end must be a contiguous int32 [G] tensor")
    G = group_end.shape[0]
    if out is None:
        out = torch.empty((G, M, N), dtype=out_dtype, device=a.device)
    _check_shape(out, (G, M, N), "out")
    if out.dtype not in OUT_DTYPES or out.stride(2) != 1:
        raise ValueError("out must be bfloat16 or float32 with unit column stride")
    if G == 0:
        return out
    nws = lib.fp8bw_grouped_wgrad_ws_bytes(M, N, K, G)
    ws = torch.empty(nws, dtype=torch.uint8, device=a.device) if nws else None
    check(lib.fp8_scaled_grouped_gemm_blockwise_wgrad(
        a.data_ptr(), a.stride(0), ra.data_ptr(), ra.stride(0), ra.stride(1), b.data_ptr(), b.stride(0),
        rb.data_ptr(), rb.stride(0), rb.stride(1), G, group_end.data_ptr(), M, N, K, out.data_ptr(),
        out.stride(1), out.stride(0), OUT_DTYPES[out.dtype], _ptr(ws), nws, _stream(a)))
    return out


def grouped_wgrad_plan(M, N, K, groups, out_dtype=torch.bfloat16):
    """How the library runs such a call (contiguous operands and outputs,
    column-major scales) on the current device: tile configuration (0: 128x128,
    1: 64x64, 3: 256x256), pieces of every group's contraction, output tiles of all
    groups, and whether one workgroup per compute unit runs them as one stream."""
    import ctypes
    info = (ctypes.c_int64 * 4)()
    check(load_library().fp8bw_grouped_wgrad_plan(M, N, K, groups, OUT_DTYPES[out_dtype], info))
    config, pieces, tiles, stream = (int(v) for v in info)
    return {"config": config, "pieces": pieces, "tiles": tiles, "stream": bool(stream)}


@_on_tensor_device
def fp8_blockwise_quant_grouped(x, transpose=False):
    """fp8_blockwise_quant(x[g], "128x128", transpose) of every matrix of x bf16
    [G, rows, cols] in one launch: (q uint8 [G, rows, cols], or [G, cols, rows]
    with transpose, recip fp32 [G, ni, nj], column-major per matrix)."""
    lib = load_library()
    _need_cuda(x)
    if x.dim() != 3 or x.stride(2) != 1 or x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16 [G, rows, cols] with unit column stride")
    G, rows, cols = x.shape
    q = torch.empty((G, cols, rows) if transpose else (G, rows, cols), dtype=torch.uint8, device=x.device)
    ni, nj = scale_grid(rows, cols, "128x128", transpose)
    recip = torch.empty((G, nj, ni), dtype=torch.float32, device=x.device).transpose(1, 2)
    if G:
        check(lib.fp8_blockwise_quant_grouped(x.data_ptr(), rows, cols, x.stride(1), x.stride(0), G,
                                              int(bool(transpose)), q.data_ptr(), q.stride(1), q.stride(0),
                                              recip.data_ptr(), 1, max(ni, 1), ni * nj, _stream(x)))
    return q, recip
