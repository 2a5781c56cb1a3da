"""Measured cases of the training-step operators around the FP8 linear: the
RMS norm that feeds it (with the residual's addition and E4M3 outputs), the
cross entropy of a linear head over a large vocabulary, and the AdamW step
over many tensors.  `run` computes them in plain torch operations, or, with
`own`, through the package's entry points, on the same inputs."""

import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 1e-12
IGNORE = -100
MASK32 = 0xFFFFFFFF


def listed():
    return [
        # Norm: one new token in front of a quantized linear (serving); a
        # ragged batch of tokens out of a wider buffer, codes and bf16 out;
        # the norm of a training forward, which writes both code layouts for
        # the linear's forward and weight gradient; its backward.
        {"name": "norm_fwd_one_token", "op": "norm", "dir": "fwd", "rows": 1, "cols": 8192,
         "residual": True, "y": False, "q": True, "qt": False, "weight": "bf16", "pad": 0},
        {"name": "norm_fwd_ragged", "op": "norm", "dir": "fwd", "rows": 777, "cols": 5136,
         "residual": True, "y": True, "q": True, "qt": False, "weight": "f32", "pad": 48},
        {"name": "norm_fwd_train", "op": "norm", "dir": "fwd", "rows": 16640, "cols": 8192,
         "residual": True, "y": False, "q": True, "qt": True, "weight": "bf16", "pad": 0},
        {"name": "norm_bwd_train", "op": "norm", "dir": "bwd", "rows": 16640, "cols": 8192,
         "residual": True, "y": False, "q": False, "qt": False, "weight": "bf16", "pad": 0},
        # Head: scoring a few tokens against a large vocabulary (the weight is
        # read once for little work); a small model's step; a step at odd
        # token and vocabulary counts; a large step.
        {"name": "head_score", "op": "head", "dir": "fwd", "tokens": 33, "vocab": 131072,
         "hidden": 5120, "ignored": 0.0},
        {"name": "head_step_small", "op": "head", "dir": "step", "tokens": 128, "vocab": 2048,
         "hidden": 512, "ignored": 0.1},
        {"name": "head_step_odd", "op": "head", "dir": "step", "tokens": 1777, "vocab": 50001,
         "hidden": 2048, "ignored": 0.25},
        {"name": "head_step_large", "op": "head", "dir": "step", "tokens": 8192, "vocab": 131072,
         "hidden": 4096, "ignored": 0.05},
        # Optimizer: a small model's many short tensors (launch and host cost);
        # odd sizes packed without gaps, so that few are aligned; a stack of
        # linear weights with 8-bit states; the same kind of stack with fp32
        # states and fp32 master weights.
        {"name": "adamw_small", "op": "adamw", "layers": 6, "d": 512, "f": 256, "param": "f32",
         "grad": "f32", "bits": 32, "master": False, "stochastic": False, "packed": False},
        {"name": "adamw_odd", "op": "adamw", "layers": 3, "d": 1023, "f": 2731, "param": "bf16",
         "grad": "f32", "bits": 8, "master": False, "stochastic": True, "packed": True},
        {"name": "adamw_8bit", "op": "adamw", "layers": 4, "d": 5120, "f": 8192, "param": "bf16",
         "grad": "bf16", "bits": 8, "master": False, "stochastic": True, "packed": False},
        {"name": "adamw_master", "op": "adamw", "layers": 4, "d": 5120, "f": 8192, "param": "bf16",
         "grad": "bf16", "bits": 32, "master": True, "stochastic": False, "packed": False},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "head", "adamw"])
    if op == "norm":
        direction = rng.choice(["fwd", "fwd", "bwd"])
        cols = 16 * _log(rng, 8, 1024)
        rows = _log(rng, 1, 16640)
        qt = direction == "fwd" and rng.random() < 0.4
        if qt:
            rows = (rows + 15) // 16 * 16
        while rows * cols > 16640 * 8192:
            rows = (rows // 2 + 15) // 16 * 16
        return {"op": "norm", "dir": direction, "rows": rows, "cols": cols,
                "residual": rng.random() < 0.7, "y": not qt and rng.random() < 0.5,
                "q": qt or rng.random() < 0.7, "qt": qt, "weight": rng.choice(["bf16", "f32"]),
                "pad": rng.choice([0, 0, 16, 48])}
    if op == "head":
        tokens, vocab, hidden = _log(rng, 1, 8192), _log(rng, 500, 131072), 64 * _log(rng, 4, 80)
        while tokens * vocab * hidden > 8192 * 131072 * 4096:
            tokens = tokens // 2
        return {"op": "head", "dir": rng.choice(["fwd", "step", "step"]), "tokens": tokens,
                "vocab": vocab, "hidden": hidden, "ignored": rng.choice([0.0, 0.1, 0.5])}
    d, f, layers = _log(rng, 64, 6000), _log(rng, 64, 9000), rng.randint(1, 8)
    while layers * d * f > 4 * 5120 * 8192:
        layers, f = max(1, layers // 2), f - f // 3
    param, bits = rng.choice(["bf16", "f32"]), rng.choice([8, 32])
    return {"op": "adamw", "layers": layers, "d": d, "f": f, "param": param,
            "grad": rng.choice(["bf16", "f32"]), "bits": bits,
            "master": param == "bf16" and rng.random() < 0.5,
            "stochastic": rng.random() < 0.5, "packed": rng.random() < 0.3}


# ---------------------------------------------------------------------------
# Inputs.

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"norm": _prepare_norm, "head": _prepare_head, "adamw": _prepare_adamw}[case["op"]](
        dict(case), gen, int(seed))


def _prepare_norm(case, gen, seed):
    rows, cols, pad = case["rows"], case["cols"], case["pad"]

    def matrix(std):
        return _normal(gen, rows, cols + pad, std=std)[:, :cols]

    weight = (1.0 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(TYPES[case["weight"]])
    st = {"case": case, "weight": weight, "eps": 1e-6}
    if case["dir"] == "fwd":
        # a residual stream grows with depth, a block's output is of order one
        st["x"] = matrix(1.0)
        st["residual"] = matrix(4.0) if case["residual"] else None
    else:
        st["s"] = matrix(4.0)
        st["rstd"] = torch.rsqrt(st["s"].float().square().mean(1) + st["eps"])
        st["dy"] = matrix(1e-3)
        st["dres"] = matrix(1e-3) if case["residual"] else None
    return st


def _prepare_head(case, gen, seed):
    T, V, K = case["tokens"], case["vocab"], case["hidden"]
    h = _normal(gen, T, K)                                   # a normed hidden state
    w = torch.empty(V, K, dtype=torch.bfloat16, device="cuda")
    for v in range(0, V, 16384):
        w[v:v + 16384] = _normal(gen, min(16384, V - v), K, std=2.0 / math.sqrt(K))
    target = torch.randint(0, V, (T,), generator=gen, device="cuda")
    if case["ignored"]:
        target[torch.rand(T, generator=gen, device="cuda") < case["ignored"]] = IGNORE
    valid = target != IGNORE
    # gradient of the mean over the tokens that count
    dloss = valid.float() / valid.sum().clamp(min=1).float()
    return {"case": case, "h": h, "w": w, "target": target, "dloss": dloss}


def _adamw_shapes(case):
    one = [case["f"] * case["d"], case["d"] * case["f"], case["d"], case["f"] + 3]
    return one * case["layers"]


def _power_of_two(e):
    """2^e as fp32, for int32 exponents in the normal range."""
    return ((e + 127) << 23).view(torch.float32)


def _blocks(t):
    """[ceil(n / 128), 128] of a vector, zeros past its end."""
    return torch.nn.functional.pad(t, (0, -t.numel() % 128)).view(-1, 128)


def _block_scale(t):
    """Power-of-two scale of each block of 128: the least that keeps |t| / scale <= 448."""
    fraction, exponent = torch.frexp(_blocks(t).abs().amax(1))
    e = exponent.to(torch.int32) - 9 + (fraction > 0.875).to(torch.int32)
    return torch.where(fraction > 0, _power_of_two(e.clamp(-126, 127)), 1.0)


def _prepare_adamw(case, gen, seed):
    numels = _adamw_shapes(case)
    gap = 1 if case["packed"] else 128
    starts, blocks, total = [], [0], 0
    for n in numels:
        starts.append(total)
        total += -(-n // gap) * gap
        blocks.append(blocks[-1] + -(-n // 128))

    def views(flat):
        return [flat[a:a + n] for a, n in zip(starts, numels)]

    def scale_views(flat):
        return [flat[a:b] for a, b in zip(blocks, blocks[1:])]

    def fresh(dtype):
        return torch.zeros(total, dtype=dtype, device="cuda")

    flat = {"param": fresh(TYPES[case["param"]]), "grad": fresh(TYPES[case["grad"]])}
    if case["master"]:
        flat["master"] = fresh(torch.float32)
    if case["bits"] == 8:
        for k in ("m", "root"):
            flat[k] = fresh(torch.uint8)
            flat[k + "_scale"] = torch.ones(blocks[-1], device="cuda")
    else:
        flat["m"], flat["v"] = fresh(torch.float32), fresh(torch.float32)
    lists = {k: scale_views(v) if k.endswith("_scale") else views(v) for k, v in flat.items()}
    for i, n in enumerate(numels):
        value = torch.randn(n, generator=gen, device="cuda").mul_(0.02)
        if case["master"]:
            lists["master"][i].copy_(value)
        lists["param"][i].copy_(value)
        # gradients of one tensor span several orders of magnitude
        size = 1e-3 * torch.exp(torch.randn(n, generator=gen, device="cuda"))
        lists["grad"][i].copy_(torch.randn(n, generator=gen, device="cuda") * size)
        m = torch.randn(n, generator=gen, device="cuda") * size * 0.3
        if case["bits"] == 8:
            for k, t in (("m", m), ("root", size)):
                scale = _block_scale(t)
                lists[k + "_scale"][i].copy_(scale)
                code = (_blocks(t) / scale[:, None]).view(-1)[:n].to(torch.float8_e4m3fn)
                lists[k][i].copy_(code.view(torch.uint8))
        else:
            lists["m"][i].copy_(m)
            lists["v"][i].copy_(size.square())
    return {"case": case, "flat": flat, "lists": lists, "seed": seed * 7919 + 11 if case["stochastic"] else None,
            "grad_scale": torch.full((1,), 0.5, device="cuda"), "step": 10, "lr": 3e-4,
            "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}


# ---------------------------------------------------------------------------
# One pass.

def run(state):
    return {"norm": _run_norm, "head": _run_head, "adamw": _run_adamw}[state["case"]["op"]](state)


def _codes_1x128(v):
    """(E4M3 codes, reciprocal scales) of fp32 rows in blocks of 128 columns."""
    rows, cols = v.shape
    b = torch.nn.functional.pad(v, (0, -cols % 128)).view(rows, -1, 128)
    s = E4M3_MAX / b.abs().amax(2).clamp(min=AMAX_FLOOR)
    q = (b * s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :cols]
    return q.to(torch.float8_e4m3fn), 1.0 / s


def _run_norm(st):
    case = st["case"]
    if case["dir"] == "bwd":
        if own:
            import blockwise_scaled_fp8_amd as fp8
            dx, dw = fp8.rms_norm_bwd(st["dy"], st["s"], st["rstd"], st["weight"], dres=st["dres"])
            return {"dx": dx, "dweight": dw}
        s_hat = st["s"].float() * st["rstd"][:, None]
        dy = st["dy"].float()
        d = dy * st["weight"].float()
        dx = st["rstd"][:, None] * (d - s_hat * (d * s_hat).mean(1, keepdim=True))
        if st["dres"] is not None:
            dx = dx + st["dres"].float()
        return {"dx": dx.to(torch.bfloat16), "dweight": (dy * s_hat).sum(0).to(st["weight"].dtype)}
    if own:
        import blockwise_scaled_fp8_amd as fp8
        o = fp8.rms_norm_fwd(st["x"], st["weight"], residual=st["residual"], eps=st["eps"],
                             y=case["y"], q=case["q"], qt=case["qt"])
        out = {"s": o.s, "rstd": o.rstd}
        if case["y"]:
            out["y"] = o.y
        if case["q"]:
            out |= {"q": o.q.view(torch.float8_e4m3fn), "recip": o.recip}
        if case["qt"]:
            out |= {"qt": o.qt.view(torch.float8_e4m3fn), "recip_t": o.recip_t}
        return out
    s = st["x"]
    if st["residual"] is not None:
        s = (s.float() + st["residual"].float()).to(torch.bfloat16)
    sf = s.float()
    rstd = 1.0 / torch.sqrt(sf.square().mean(1) + st["eps"])
    v = sf * rstd[:, None] * st["weight"].float()
    out = {"s": s, "rstd": rstd}
    if case["y"]:
        out["y"] = v.to(torch.bfloat16)
    if case["q"]:
        out["q"], out["recip"] = _codes_1x128(v)
    if case["qt"]:
        out["qt"], out["recip_t"] = _codes_1x128(v.t().contiguous())
    return out


def _run_head(st):
    h, w, target, dloss = st["h"], st["w"], st["target"], st["dloss"]
    step = st["case"]["dir"] == "step"
    if own:
        import blockwise_scaled_fp8_amd as fp8
        loss, lse = fp8.linear_xent_fwd(h, w, target, ignore_index=IGNORE)
        out = {"loss": loss, "lse": lse}
        if step:
            out["dh"], out["dw"] = fp8.linear_xent_bwd(dloss, h, w, target, lse, ignore_index=IGNORE)
        return out
    valid = target != IGNORE
    at = target.clamp(min=0)[:, None]
    hf, wf = h.float(), w.float()
    logits = hf @ wf.t()
    top = logits.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    loss = torch.where(valid, (lse - logits.gather(1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": lse[:, 0]}
    if step:
        g = logits.sub_(lse).exp_()
        g.scatter_add_(1, at, torch.full_like(lse, -1.0))
        g.mul_((dloss * valid)[:, None])
        out["dh"] = (g @ wf).to(torch.bfloat16)
        out["dw"] = (g.t() @ hf).to(torch.bfloat16)
    return out


def _mix(x):
    """A 32-bit mixing function of int64 values (only their low 32 bits count)."""
    x = x & MASK32
    x = ((x ^ (x >> 16)) * 0x6A09E667) & MASK32
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & MASK32
    return x ^ (x >> 16)


def _random_bits(seed, ordinal, n):
    """Three random 16-bit numbers for each of a tensor's n elements."""
    key = _mix(seed + 0x9E3779B9 * (ordinal + 1)) + (seed >> 32)
    bits = _mix(torch.arange(n, device="cuda") + key)
    return bits & 0xFFFF, bits >> 16, ((bits * 0x9E3779B9) & MASK32) >> 16


def _to_e4m3(t, scale, random, keep_positive):
    """t / scale on the E4M3 grid, rounded up or down by 16 random bits or to nearest."""
    y = (_blocks(t) / scale[:, None]).view(-1)[:t.numel()]
    size = y.abs()
    ulp = _power_of_two((torch.frexp(size)[1].to(torch.int32) - 1).clamp(min=-6) - 3)
    steps = size / ulp
    steps = torch.round(steps) if random is None else torch.floor(steps + random.float() / 65536)
    size_on_grid = steps * ulp
    if keep_positive:
        size_on_grid = torch.where(size > 0, size_on_grid.clamp(min=2.0 ** -9), size_on_grid)
    return torch.copysign(size_on_grid, y).to(torch.float8_e4m3fn).view(torch.uint8)


def _run_adamw(st):
    case, lists = st["case"], st["lists"]
    eight = case["bits"] == 8
    if own:
        import blockwise_scaled_fp8_amd as fp8
        fp8.adamw_step(lists["param"], lists["grad"], lists["m"], lists["root" if eight else "v"],
                       step=st["step"], lr=st["lr"], beta1=st["beta1"], beta2=st["beta2"],
                       eps=st["eps"], weight_decay=st["weight_decay"],
                       exp_avg_scales=lists.get("m_scale"), root_scales=lists.get("root_scale"),
                       masters=lists.get("master"), grad_scale=st["grad_scale"], seed=st["seed"])
    else:
        for i in range(len(lists["param"])):     # one tensor after the other, as a plain optimizer
            _plain_adamw(st, lists, i, eight)
    out = dict(st["flat"])
    del out["grad"]
    if eight:
        out["m"] = out["m"].view(torch.float8_e4m3fn)
        out["root"] = out["root"].view(torch.float8_e4m3fn)
    return out


def _plain_adamw(st, lists, i, eight):
    param = lists["param"][i]
    master = lists["master"][i] if "master" in lists else param
    n, b1, b2 = param.numel(), st["beta1"], st["beta2"]
    low, high, last = (None, None, None) if st["seed"] is None else _random_bits(st["seed"], i, n)
    g = lists["grad"][i].float() * st["grad_scale"]
    if eight:
        m, root = (lists[k][i].view(torch.float8_e4m3fn).float()
                   * lists[k + "_scale"][i].repeat_interleave(128)[:n] for k in ("m", "root"))
        v = root * root
    else:
        m, v = lists["m"][i], lists["v"][i]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    root = torch.sqrt(v)
    p = master.float() * (1 - st["lr"] * st["weight_decay"])
    denom = root * (1 / math.sqrt(1 - b2 ** st["step"])) + st["eps"]
    p = p - m / denom * (st["lr"] / (1 - b1 ** st["step"]))
    if eight:
        for k, t, random, keep in (("m", m, low, False), ("root", root, high, True)):
            scale = _block_scale(t)
            lists[k + "_scale"][i].copy_(scale)
            lists[k][i].copy_(_to_e4m3(t, scale, random, keep))
    else:
        lists["m"][i].copy_(m)
        lists["v"][i].copy_(v)
    master.copy_(p)
    if "master" not in lists and param.dtype == torch.bfloat16 and last is not None:
        # to bf16 by 16 random bits: added below the cut, then cut off
        bits = p.view(torch.int32).long() + last
        param.copy_(((bits & 0xFFFF0000) - ((bits & 0x80000000) << 1)).to(torch.int32).view(torch.float32))
    else:
        param.copy_(p)


# ---------------------------------------------------------------------------
# What a pass has to move and compute.

def work(case):
    if case["op"] == "norm":
        n, cols, rows = case["rows"] * case["cols"], case["cols"], case["rows"]
        wb = 2 if case["weight"] == "bf16" else 4
        blocks = rows * -(-cols // 128)
        if case["dir"] == "bwd":
            return {"bytes": n * (6 + 2 * case["residual"]) + 4 * rows + 2 * wb * cols, "flops": 10 * n}
        moved = n * (2 + 4 * case["residual"] + 2 * case["y"] + case["q"] + case["qt"])
        moved += 4 * rows + wb * cols + 4 * blocks * case["q"] + 4 * cols * -(-rows // 128) * case["qt"]
        return {"bytes": moved, "flops": 8 * n}
    if case["op"] == "head":
        T, V, K = case["tokens"], case["vocab"], case["hidden"]
        step = case["dir"] == "step"
        # products only: the logits, and for a step the two gradients
        return {"bytes": 2 * (T * K + V * K) * (2 if step else 1) + 8 * T + 8 * T + 4 * T * step,
                "flops": (6 if step else 2) * T * V * K}
    n = sum(_adamw_shapes(case))
    p, g = (2 if case[k] == "bf16" else 4 for k in ("param", "grad"))
    states = 4 + 16 / 128 if case["bits"] == 8 else 16
    weights = 8 + p if case["master"] else 2 * p
    return {"bytes": n * (weights + g + states), "flops": 16 * n}


# ---------------------------------------------------------------------------
# The same from the definitions in 64 bits.  What is held in 8 or 16 bits by a
# rounding up or down at random, or in codes, is given as the value that is
# rounded.

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "head": _exact_head, "adamw": _exact_adamw}[case["op"]](st)


def _exact_scaled(v):
    """Rows of v in units of their blocks' E4M3 scales, and the reciprocals."""
    rows, cols = v.shape
    q, recip = torch.empty_like(v), []
    for c in range(0, cols, 128):
        block = v[:, c:c + 128]
        recip.append(block.abs().amax(1).clamp(min=AMAX_FLOOR) / E4M3_MAX)
        q[:, c:c + 128] = block / recip[-1][:, None]
    return q, torch.stack(recip, 1)


def _exact_norm(st):
    case, w = st["case"], st["weight"].double()
    if case["dir"] == "bwd":
        s, dy, rstd = st["s"].double(), st["dy"].double(), st["rstd"].double()[:, None]
        inner = (dy * w * s).sum(1, keepdim=True) / case["cols"]
        dx = dy * w * rstd - s * rstd ** 3 * inner
        if st["dres"] is not None:
            dx += st["dres"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc,ro->c", dy, s, rstd)}
    s = st["x"].double()
    if st["residual"] is not None:
        # the sum is exact in 32 bits or rounds there first, as it is defined: to bf16
        s = (st["x"].float() + st["residual"].float()).to(torch.bfloat16).double()
    rstd = (torch.linalg.vector_norm(s, dim=1) ** 2 / case["cols"] + st["eps"]) ** -0.5
    v = s * rstd[:, None] * w
    out = {"s": s, "rstd": rstd}
    if case["y"]:
        out["y"] = v
    if case["q"]:
        out["q"], out["recip"] = _exact_scaled(v)
    if case["qt"]:
        out["qt"], out["recip_t"] = _exact_scaled(v.t().contiguous())
    return out


def _exact_head(st):
    h, w, target, dloss = st["h"].double(), st["w"].double(), st["target"], st["dloss"].double()
    T = h.shape[0]
    step = st["case"]["dir"] == "step"
    loss, lse = torch.zeros(T, dtype=torch.float64, device="cuda"), torch.empty(T, dtype=torch.float64, device="cuda")
    dh, dw = torch.zeros_like(h), torch.zeros_like(w) if step else None
    for t0 in range(0, T, 1024):
        rows = slice(t0, min(T, t0 + 1024))
        z = torch.mm(h[rows], w.t())
        lse[rows] = torch.logsumexp(z, 1)
        own_target = target[rows]
        counts = (own_target != IGNORE).nonzero()[:, 0]
        loss[rows][counts] = lse[rows][counts] - z[counts, own_target[counts]]
        if step:
            prob = torch.softmax(z, 1)
            prob[counts, own_target[counts]] -= 1.0
            weight = torch.zeros_like(lse[rows])
            weight[counts] = dloss[rows][counts]
            prob *= weight[:, None]
            dh[rows] = torch.mm(prob, w)
            dw += torch.mm(prob.t().contiguous(), h[rows])
    out = {"loss": loss, "lse": lse}
    if step:
        out |= {"dh": dh, "dw": dw}
    return out


def _exact_adamw(st):
    case, lists = st["case"], st["lists"]
    eight, t = case["bits"] == 8, st["step"]
    out = {k: v.double() for k, v in st["flat"].items() if k != "grad" and v.dtype != torch.uint8}
    if eight:
        out |= {k: st["flat"][k].view(torch.float8_e4m3fn).double() for k in ("m", "root")}
    for i, param in enumerate(lists["param"]):
        n = param.numel()
        at = slice(param.storage_offset(), param.storage_offset() + n)
        g = lists["grad"][i].double() * float(st["grad_scale"])
        if eight:
            scale = {k: lists[k + "_scale"][i].double().repeat_interleave(128)[:n] for k in ("m", "root")}
            m = out["m"][at] * scale["m"]
            v = (out["root"][at] * scale["root"]) ** 2
        else:
            m, v = out["m"][at], out["v"][at]
        m = m + (1 - st["beta1"]) * (g - m)
        v = v + (1 - st["beta2"]) * (g * g - v)
        m_hat, v_hat = m / (1 - st["beta1"] ** t), v / (1 - st["beta2"] ** t)
        kept = "master" if case["master"] else "param"
        p = out[kept][at]
        p = p - st["lr"] * (m_hat / (v_hat.sqrt() + st["eps"]) + st["weight_decay"] * p)
        out[kept][at] = p
        out["param"][at] = p
        if eight:
            first = lists["m_scale"][i].storage_offset()
            for k, value in (("m", m), ("root", v.sqrt())):
                top = _blocks(value).abs().amax(1)
                new = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))
                new = torch.where(top > 0, new, torch.ones_like(new))
                out[k + "_scale"][first:first + new.numel()] = new
                out[k][at] = value / new.repeat_interleave(128)[:n]
        else:
            out["m"][at], out["v"][at] = m, v
    return out
