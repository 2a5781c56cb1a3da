"""Plain 64-bit implementations of the mixture-of-experts operators (oracle;
test infrastructure only): slots sorted by expert, rows gathered and joined,
the gated activation and its gradient, grouped weight gradients.  Written from
the formulas, with numpy, without the GPU path's code."""

import numpy as np

from . import e4m3, gemm


def rows_bound(tokens, topk, experts, align):
    """The most rows that any assignment fills: as many experts as there can be
    start a block of `align` rows, the other slots fill further whole blocks."""
    n = tokens * topk
    filled = min(experts, n)
    return align * (filled + (n - filled) // align)


def sort(expert, experts, align, rows):
    """(row [tokens, topk], source [rows], group_end [experts]), one slot after
    the other."""
    expert = np.asarray(expert)
    members = [[] for _ in range(experts)]
    for i, e in enumerate(expert.reshape(-1)):
        if 0 <= e < experts:
            members[e].append(i)
    row = np.full(expert.size, -1, np.int64)
    source = np.full(rows, -1, np.int64)
    ends, at = [], 0
    for slots in members:
        for r, i in enumerate(slots, at):
            row[i], source[r] = r, i
        at += -(-len(slots) // align) * align
        ends.append(at)
    return row.reshape(expert.shape), source, np.array(ends, np.int64)


def gather(x, source, topk, weight=None):
    """v[r] = weight[source[r]] x[source[r] // topk], zeros without a slot."""
    x = np.asarray(x, np.float64)
    v = np.zeros((len(source), x.shape[1]))
    for r, i in enumerate(source):
        if i >= 0:
            v[r] = x[i // topk] * (1.0 if weight is None else float(np.asarray(weight, np.float64).reshape(-1)[i]))
    return v


def combine(y, row, weight=None):
    """(out, sum of the terms' magnitudes): out[t] = sum_j weight[t, j] y[row[t, j]]."""
    y = np.asarray(y, np.float64)
    out = np.zeros((row.shape[0], y.shape[1]))
    size = np.zeros_like(out)
    for t, js in enumerate(row):
        for j, r in enumerate(js):
            if r >= 0:
                part = y[r] * (1.0 if weight is None else float(weight[t, j]))
                out[t] += part
                size[t] += np.abs(part)
    return out, size


def combine_dweight(dout, y, row):
    """(dweight, sum of the products' magnitudes)."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    dw = np.zeros(row.shape)
    size = np.zeros(row.shape)
    for t, js in enumerate(row):
        for j, r in enumerate(js):
            if r >= 0:
                dw[t, j] = (dout[t] * y[r]).sum()
                size[t, j] = np.abs(dout[t] * y[r]).sum()
    return dw, size


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def swiglu(h):
    """v = g sigmoid(g) u of h = [g | u]."""
    g, u = np.split(np.asarray(h, np.float64), 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_grad(dy, h):
    """([dg | du], the same with every term's magnitude) of sum(dy * swiglu(h))."""
    g, u = np.split(np.asarray(h, np.float64), 2, axis=1)
    dy = np.asarray(dy, np.float64)
    s, away = sigmoid(g), sigmoid(-g)          # 1 - s without cancellation
    slope = s + g * s * away
    terms = s + np.abs(g) * s * away
    return (np.concatenate([dy * u * slope, dy * g * s], 1),
            np.concatenate([np.abs(dy * u) * terms, np.abs(dy * g * s)], 1))


def halves_values(codes, recip):
    """What codes with a scale per 1x128 block of each half stand for."""
    v = e4m3.decode(codes).astype(np.float64)
    ffn = v.shape[1] // 2
    block = np.arange(ffn) // 128
    return v * np.asarray(recip, np.float64)[:, np.concatenate([block, -(-ffn // 128) + block])]


def grouped_wgrad(a, ra, b, rb, group_end):
    """([G, M, N], error scale): each group's blocks of 128 of the contraction."""
    M, K = a.shape
    out = np.zeros((len(group_end), M, b.shape[0]))
    size = np.zeros_like(out)
    first = 0
    for g, end in enumerate(group_end):
        begin, last = min(first // 128, K // 128), min(end // 128, K // 128)
        if last > begin:
            k, kb = slice(begin * 128, last * 128), slice(begin, last)
            out[g], size[g] = gemm.blockwise_gemm(a[:, k], ra[:, kb], b[:, k], rb[:, kb], "1x128", with_bound=True)
        first = end
    return out, size
