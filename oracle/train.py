"""Plain 64-bit implementations of the operators around the linear in a
training step (oracle; test infrastructure only): RMS norm with the residual's
addition, softmax cross entropy of a linear head, AdamW with fp32 or 8-bit
block-scaled states.  Written from the formulas, with numpy, without the GPU
path's code."""

import numpy as np

from . import e4m3, quant


# ---------------------------------------------------------------------------
# RMS norm.

def residual_sum(x, residual):
    """s = bf16(x + residual) of bf16-valued arrays, as float64.  Two bf16
    values add exactly in float64; fp32 rounds the sum once before bf16 does."""
    s32 = (np.asarray(x, np.float64) + np.asarray(residual, np.float64)).astype(np.float32)
    return e4m3.rne_bf16(s32).astype(np.float64)


def rms_norm_fwd(s, weight, eps):
    """(v, rstd): v = s rstd weight, rstd = (mean s^2 + eps)^-1/2 per row."""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + eps)
    return s * rstd[:, None] * np.asarray(weight, np.float64), rstd


def rms_norm_bwd(dy, s, weight, eps, dres=None):
    """(dx, dweight) of rms_norm_fwd, from the quotient rule."""
    dy, s, weight = (np.asarray(a, np.float64) for a in (dy, s, weight))
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    d = dy * weight
    dx = d * rstd - s * rstd ** 3 * (d * s).mean(axis=1, keepdims=True)
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, (dy * s * rstd).sum(axis=0)


def blocks_1x128(v):
    """(v in units of its blocks' E4M3 scales, reciprocals), blocks of 128
    columns, a ragged last block over its own columns."""
    q, recip = np.empty_like(v), []
    for c in range(0, v.shape[1], 128):
        amax = np.maximum(np.abs(v[:, c:c + 128]).max(axis=1), float(quant.EPS))
        recip.append(amax / 448.0)
        q[:, c:c + 128] = v[:, c:c + 128] / recip[-1][:, None]
    return q, np.stack(recip, axis=1)


# ---------------------------------------------------------------------------
# Linear cross entropy.

def linear_xent(h, w, target, ignore_index=-100, dloss=None):
    """(loss, lse) per token, and with dloss also (dh, dw)."""
    h, w, target = np.asarray(h, np.float64), np.asarray(w, np.float64), np.asarray(target)
    z = h @ w.T
    top = z.max(axis=1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(z - top).sum(axis=1))
    counts = target != ignore_index
    known = counts & (target >= 0) & (target < w.shape[0])
    t = np.arange(len(target))
    loss = np.zeros(len(target))
    loss[known] = lse[known] - z[t[known], target[known]]
    loss[counts & ~known] = np.nan
    if dloss is None:
        return loss, lse
    g = np.exp(z - lse[:, None])
    g[t[known], target[known]] -= 1.0
    g *= np.where(known, np.asarray(dloss, np.float64), 0.0)[:, None]
    return loss, lse, g @ w, g.T @ h


# ---------------------------------------------------------------------------
# AdamW.

def adamw(p, g, m, v, *, step, lr, beta1, beta2, eps, weight_decay):
    """(p, m, v) after one step, float64."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * (mh / (np.sqrt(vh) + eps) + weight_decay * p), m, v


def state_scales(x):
    """Power-of-two scale per 128 elements: the least 2^e with |x| <= 448 2^e,
    1 for a block of zeros."""
    x = np.pad(np.abs(np.asarray(x, np.float64)), (0, -len(x) % 128)).reshape(-1, 128).max(axis=1)
    out = np.ones(len(x))
    for i, a in enumerate(x):
        if a > 0:
            e = int(np.floor(np.log2(a / 448.0))) - 1
            while a > 448.0 * 2.0 ** e:
                e += 1
            out[i] = 2.0 ** max(e, -126)
    return out


def mix32(x):
    """The 32-bit mixing function of the random bits (int arrays or ints)."""
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    m, u = np.uint64(0xFFFFFFFF), np.uint64
    x = ((x ^ (x >> u(16))) * u(0x6A09E667)) & m
    x = ((x ^ (x >> u(15))) * u(0xBB67AE85)) & m
    return x ^ (x >> u(16))


def random_bits(seed, ordinal, n):
    """(for m, for the root, for a bf16 parameter): 16 bits per element each."""
    u = np.uint64
    key = (int(mix32((seed & 0xFFFFFFFF) + 0x9E3779B9 * (ordinal + 1))) + (seed >> 32)) & 0xFFFFFFFF
    h = mix32(np.arange(n, dtype=np.uint64) + u(key))
    return h & u(0xFFFF), h >> u(16), ((h * u(0x9E3779B9)) & u(0xFFFFFFFF)) >> u(16)


def e4m3_neighbours(y):
    """(down, up, spacing): the E4M3 grid's values around |y| <= 448, towards
    and away from zero, and their distance."""
    a = np.abs(np.asarray(y, np.float64))
    e = np.full(a.shape, -6.0)
    nz = a >= 2.0 ** -6
    e[nz] = np.floor(np.log2(a[nz]))
    e = np.where(2.0 ** e > a, np.maximum(e - 1, -6), e)     # log2 rounded up
    ulp = 2.0 ** (e - 3)
    down = np.floor(a / ulp) * ulp
    return down, np.where(a == down, down, down + ulp), ulp


def e4m3_stochastic(y, r16):
    """|y| rounded up with probability remainder / spacing, in units of 2^-16."""
    down, _, ulp = e4m3_neighbours(y)
    frac = (np.abs(y) - down) / ulp
    out = down + np.where(frac + np.asarray(r16, np.float64) / 65536.0 >= 1.0, ulp, 0.0)
    return np.copysign(out, y)
