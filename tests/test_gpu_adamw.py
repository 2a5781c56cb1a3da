"""The multi-tensor AdamW step on the GPU against the 64-bit oracle.

Tolerances (u = 2^-24): m and v take three roundings each, within 4 u of the
magnitudes added; the step has about 12 (two of them hardware forms of 1 ulp),
within 32 u of itself, plus 3 u of p.  Codes: with the scale given, the value
that the definition rounds to, except where the remainder plus the random
number is within 2^-12 and the value's own tolerance of the next step, or (to
nearest) of a tie.  bf16 parameters: half their spacing."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import e4m3, metrics, train
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(step=7, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
# one element; around a thread's 8, a block's 128, a workgroup's 2048; odd and long
NUMELS = [1, 7, 8, 9, 127, 128, 129, 2047, 2048, 2049, 100003]


def _f64(t):
    return t.detach().cpu().double().numpy()


def _tensor(n, seed, gpu, param, grad, bits, master, offset=0):
    """One tensor's buffers on the GPU, `offset` elements into wider ones."""
    g = torch.Generator().manual_seed(seed)

    def put(t):
        wide = torch.full((n + offset + 3,), 3, dtype=t.dtype)
        wide[offset:offset + n] = t
        return wide.to(gpu)[offset:offset + n]
    size = 1e-3 * torch.exp(torch.randn(n, generator=g))
    p = torch.randn(n, generator=g) * 0.05
    d = {"grad": put((torch.randn(n, generator=g) * size).to(grad)), "param": put(p.to(param))}
    m = torch.randn(n, generator=g) * size * 0.3
    if master:
        d["master"] = put(p)
    if bits == 8:
        for k, t in (("m", m), ("root", size)):
            s = train.state_scales(t.numpy())
            y = t.numpy() / np.repeat(s, 128)[:n]
            d[k] = put(torch.from_numpy(e4m3.encode_rne(y)))
            d[k + "_scale"] = torch.from_numpy(s).float().to(gpu)
    else:
        d["m"], d["v"] = put(m), put(size * size)
    return d


def _call(ds, bits, seed, grad_scale=None, **hyper):
    fp8.adamw_step([d["param"] for d in ds], [d["grad"] for d in ds], [d["m"] for d in ds],
                   [d["root" if bits == 8 else "v"] for d in ds],
                   exp_avg_scales=[d["m_scale"] for d in ds] if bits == 8 else None,
                   root_scales=[d["root_scale"] for d in ds] if bits == 8 else None,
                   masters=[d.get("master") for d in ds], grad_scale=grad_scale, seed=seed,
                   **{**HYPER, **hyper})


def _state(d, bits):
    """(m, v) before the step, float64."""
    if bits == 32:
        return _f64(d["m"]), _f64(d["v"])
    n = d["m"].numel()
    m, r = (e4m3.decode(d[k].cpu().numpy()) * np.repeat(_f64(d[k + "_scale"]), 128)[:n] for k in ("m", "root"))
    return m, r * r


def _check_codes(code, scale, value, tol, r16, keep, what):
    n = len(value)
    near = [train.state_scales(value * (1 + d)) for d in (-8 * U, 0.0, 8 * U)]
    assert np.all([s in (a, b, c) for s, a, b, c in zip(scale, *near)]), what + " scale"
    y = np.clip(value / np.repeat(scale, 128)[:n], -448, 448)
    down, _, ulp = train.e4m3_neighbours(y)
    frac = (np.abs(y) - down) / ulp
    zone = 2.0 ** -12 + tol / np.repeat(scale, 128)[:n] / ulp
    if r16 is None:
        want, sure = down + np.where(frac > 0.5, ulp, 0.0), np.abs(frac - 0.5) > zone
    else:
        total = frac + r16.astype(np.float64) / 65536
        want, sure = down + np.where(total >= 1, ulp, 0.0), (np.abs(total - 1) > zone) & (frac < 1 - zone) & (frac > zone)
    if keep:
        want = np.where(np.abs(y) > 0, np.maximum(want, 2.0 ** -9), want)
    got = e4m3.decode(code)
    assert np.array_equal(np.abs(got)[sure], want[sure]), what
    # where the last bits decide, one of the two neighbours
    assert np.all((np.abs(got) >= down - ulp) & (np.abs(got) <= np.maximum(down + 2 * ulp, 2.0 ** -9))), what
    assert np.all((got == 0) | (np.sign(got) == np.sign(y)) | ~sure), what


def _check(before, d, ordinal, bits, seed, scale=1.0, **hyper):
    hyper = {**HYPER, **hyper}
    b1, b2, lr = hyper["beta1"], hyper["beta2"], hyper["lr"]
    n = d["param"].numel()
    m0, v0 = before["m64"], before["v64"]
    g, p0 = _f64(before["grad"]) * scale, _f64(before.get("master", before["param"]))
    p, m, v = train.adamw(p0, g, m0, v0, **hyper)
    m_tol = 4 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) + 1e-44
    v_tol = 4 * U * v + 1e-44
    r = (None,) * 3 if seed is None else train.random_bits(seed, ordinal, n)
    if bits == 32:
        assert np.all(np.abs(_f64(d["m"]) - m) <= m_tol) and np.all(np.abs(_f64(d["v"]) - v) <= v_tol)
    else:
        _check_codes(d["m"].cpu().numpy(), _f64(d["m_scale"]), m, m_tol, r[0], False, "m")
        _check_codes(d["root"].cpu().numpy(), _f64(d["root_scale"]), np.sqrt(v), 4 * U * np.sqrt(v), r[1], True, "root")
    step = np.abs(p - p0 * (1 - lr * hyper["weight_decay"]))
    bias = (1 - b1 ** hyper["step"], np.sqrt(1 - b2 ** hyper["step"]))
    # a rounding of m moves the step by m_tol over the denominator
    p_tol = 32 * U * step + 3 * U * np.abs(p0) + lr * m_tol / bias[0] / (np.sqrt(v) / bias[1] + hyper["eps"])
    kept = _f64(d.get("master", d["param"]))
    if "master" in d:
        assert np.all(np.abs(kept - p) <= p_tol)
        assert torch.equal(d["param"], d["master"].bfloat16())
    elif d["param"].dtype == torch.float32:
        assert np.all(np.abs(kept - p) <= p_tol)
    elif seed is None:
        assert np.all(np.abs(kept - p) <= p_tol + metrics.bf16_ulp(np.abs(p) + p_tol) / 2)
    else:
        # towards zero, or one bf16 step away from it if the remainder and the random number carry
        p32 = p.astype(np.float32)
        cut = (p32.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
        ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(cut), 2.0 ** -126))) - 7)
        total = (np.abs(p) - np.abs(cut)) / ulp + r[2].astype(np.float64) / 65536
        sure = np.abs(total - 1) > p_tol / ulp + 2.0 ** -12
        want = np.abs(cut) + np.where(total >= 1, ulp, 0.0)
        assert np.array_equal(np.abs(kept)[sure], want[sure])
        assert np.all(np.abs(kept - p) <= ulp + p_tol)


def _copy(ds, bits):
    out = []
    for d in ds:
        c = {k: t.clone() for k, t in d.items()}
        c["m64"], c["v64"] = _state(d, bits)
        out.append(c)
    return out


@pytest.mark.parametrize("seed", [None, 987654321987654321])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kind", ["bf16", "f32", "master", "mixed"])
def test_step(gpu, kind, bits, seed):
    types = {"bf16": (torch.bfloat16, torch.bfloat16), "f32": (torch.float32, torch.float32),
             "master": (torch.bfloat16, torch.float32), "mixed": (torch.float32, torch.bfloat16)}[kind]
    # every length twice: aligned, and at an offset that aligns nothing
    ds = [_tensor(n, 31 * n + off, gpu, *types, bits, kind == "master", off) for n in NUMELS for off in (0, 3)]
    scale = torch.full((1,), 0.5, device=gpu)
    before = _copy(ds, bits)
    say("adamw", kind, bits, seed)
    _call(ds, bits, seed, grad_scale=scale)
    torch.cuda.synchronize()
    for i, (b, d) in enumerate(zip(before, ds)):
        assert torch.equal(b["grad"], d["grad"])
        _check(b, d, i, bits, seed, scale=0.5)


def test_many_tensors_and_long_launches(gpu):
    """More tensors than one launch takes, one long enough for several runs a
    workgroup; empty ones between; random numbers go by the tensor's place."""
    numels = [257] * 43 + [0, 1, 0] + [(1 << 23) + 77]
    ds = [_tensor(n, i, gpu, torch.bfloat16, torch.bfloat16, 8, False) for i, n in enumerate(numels)]
    before = _copy(ds, 8)
    say("adamw many tensors")
    _call(ds, 8, 5)
    for i, (b, d) in enumerate(zip(before, ds)):
        if d["param"].numel():
            _check(b, d, i, 8, 5)


def test_neighbours_are_untouched(gpu):
    """Writes stay inside the tensors of a packed buffer."""
    for bits in (8, 32):
        flat = {k: torch.full((5000,), 2, dtype=t, device=gpu) for k, t in
                (("param", torch.bfloat16), ("grad", torch.bfloat16), ("m", torch.uint8 if bits == 8 else torch.float32),
                 ("v", torch.uint8 if bits == 8 else torch.float32))}
        old = {k: t.clone() for k, t in flat.items()}
        at = slice(13, 13 + 2101)
        scales = [torch.ones(17, device=gpu) for _ in range(2)] if bits == 8 else [None, None]
        say("adamw canary", bits)
        fp8.adamw_step([flat["param"][at]], [flat["grad"][at]], [flat["m"][at]], [flat["v"][at]],
                       exp_avg_scales=[scales[0]] if bits == 8 else None,
                       root_scales=[scales[1]] if bits == 8 else None, seed=1, **HYPER)
        for k in flat:
            outside = torch.ones(5000, dtype=torch.bool, device=gpu)
            outside[at] = False
            assert torch.equal(flat[k][outside], old[k][outside]), (bits, k)


def test_zero_and_vanishing_states(gpu):
    """From zero codes and gradients nothing moves but the decay; a root far
    below its block's largest keeps a code, so no step explodes."""
    n = 256
    z = dict(dtype=torch.uint8, device=gpu)
    d = {"param": torch.ones(n, device=gpu), "grad": torch.zeros(n, device=gpu), "m": torch.zeros(n, **z),
         "root": torch.zeros(n, **z), "m_scale": torch.zeros(2, device=gpu), "root_scale": torch.zeros(2, device=gpu)}
    say("adamw zero states")
    _call([d], 8, None)
    assert torch.allclose(d["param"], torch.full_like(d["param"], 1 - 1e-3)) and not d["m"].any() and not d["root"].any()
    assert bool((d["m_scale"] == 1).all()) and bool((d["root_scale"] == 1).all())
    d["grad"][0], d["grad"][1:] = 1e4, 1e-6
    for seed in (None, 3):
        _call([d], 8, seed)
        assert bool((d["root"][1:128] >= 1).all())
    d["grad"].zero_()
    p = d["param"].clone()
    _call([d], 8, 4, weight_decay=0.0)
    assert float((d["param"] - p).abs().max()) < 0.1   # lr times at most ten


def test_random_rounding_follows_a_slow_average(gpu):
    """v's average with beta2 = 0.999 reaches the gradient's square from 4
    times that; rounded to nearest its 8-bit root would never leave."""
    n = 1 << 16
    start = {"param": torch.zeros(n, device=gpu), "grad": torch.full((n,), 1e-3, device=gpu),
             "m": torch.zeros(n, dtype=torch.uint8, device=gpu), "m_scale": torch.ones(n // 128, device=gpu)}
    root = torch.full((n,), 2e-3)
    s = train.state_scales(root.numpy())
    start["root"] = torch.from_numpy(e4m3.encode_rne(root.numpy() / np.repeat(s, 128))).to(gpu)
    start["root_scale"] = torch.from_numpy(s).float().to(gpu)
    say("adamw slow average")
    means = {}
    for how in ("random", "nearest"):
        d = {k: t.clone() for k, t in start.items()}
        for step in range(1, 501):
            _call([d], 8, step if how == "random" else None, beta2=0.999, step=step)
        means[how] = float((_state(d, 8)[1]).mean())
    v = 4e-6
    v = 1e-6 + (v - 1e-6) * 0.999 ** 500
    # the mean of 65536 independent roundings; each wanders by tens of percent
    # (and E[root^2] exceeds E[root]^2 by that variance)
    assert abs(means["random"] / v - 1) < 0.25
    assert means["nearest"] / v > 1.25


def test_equal_arguments_give_equal_bits(gpu):
    ds = [_tensor(n, n, gpu, torch.bfloat16, torch.bfloat16, 8, False) for n in (5000, 129)]
    twin = [{k: t.clone() for k, t in d.items()} for d in ds]
    other = [{k: t.clone() for k, t in d.items()} for d in ds]
    say("adamw repeats")
    _call(ds, 8, 77)
    _call(twin, 8, 77)
    _call(other, 8, 78)
    for a, b, c in zip(ds, twin, other):
        assert all(torch.equal(a[k], b[k]) for k in a)
        assert not torch.equal(a["m"], c["m"])


def test_subnormal_second_moments(gpu):
    """Gradients of 1e-20, whose squares are subnormal: the root still comes
    out, within half a code (2^-4) and the subnormal's own rounding (2^-11)."""
    n = 300
    z = dict(dtype=torch.uint8, device=gpu)
    d = {"param": torch.zeros(n, device=gpu), "grad": torch.full((n,), 1e-20, device=gpu), "m": torch.zeros(n, **z),
         "root": torch.zeros(n, **z), "m_scale": torch.ones(3, device=gpu), "root_scale": torch.ones(3, device=gpu)}
    d["grad"][256:] = 1.0
    d["grad"][257] = 1e-20          # next to a large one: the smallest code
    say("adamw subnormal moments")
    _call([d], 8, None)
    root = e4m3.decode(d["root"].cpu().numpy()) * np.repeat(_f64(d["root_scale"]), 128)[:n]
    want = np.sqrt((1 - HYPER["beta2"]) * _f64(d["grad"]) ** 2)
    sure = np.arange(n) != 257
    assert np.all(np.abs(root - want)[sure] <= (2.0 ** -4 + 2.0 ** -11) * want[sure])
    assert int(d["root"][257]) == 1 and bool(d["param"].isfinite().all())
