"""Measured cases of the operators of an FP8 mixture-of-experts layer around
the grouped GEMM: tokens sorted by expert and gathered into the GEMM's operand
codes, the experts' rows joined again with the router's weights (and the
gradients of both), the gated activation between the two products with 8-bit
checkpoints for its backward, and the grouped weight gradient.  `run` computes
them in plain torch operations, or, with `own`, through the package's entry
points, on the same inputs."""

import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 1e-12


def listed():
    return [
        # Tokens to experts: one token of a decoding step against many experts
        # (codes for the quantized products); a ragged batch with padding
        # tokens out of a wider buffer, bf16 and codes; a training batch, each
        # expert's rows padded to whole blocks of 128 and both code layouts
        # written (the product's and the weight gradient's).
        {"name": "route_one_token", "op": "route", "tokens": 1, "topk": 8, "experts": 128, "cols": 5120,
         "align": 1, "y": False, "q": True, "qt": False, "dropped": 0.0, "pad": 0},
        {"name": "route_ragged", "op": "route", "tokens": 777, "topk": 6, "experts": 60, "cols": 2064,
         "align": 1, "y": True, "q": True, "qt": False, "dropped": 0.15, "pad": 48},
        {"name": "route_train", "op": "route", "tokens": 16640, "topk": 2, "experts": 16, "cols": 8192,
         "align": 128, "y": False, "q": True, "qt": True, "dropped": 0.0, "pad": 0},
        # Experts back to tokens: the same decoding step; a training forward;
        # its backward, which writes the codes of both products that read the
        # gradient, and the gradient of the router's weights.
        {"name": "join_one_token", "op": "join", "dir": "fwd", "tokens": 1, "topk": 8, "experts": 128,
         "cols": 5120, "align": 1, "weighted": True, "dropped": 0.0, "pad": 0},
        {"name": "join_train", "op": "join", "dir": "fwd", "tokens": 16640, "topk": 2, "experts": 16,
         "cols": 8192, "align": 128, "weighted": True, "dropped": 0.0, "pad": 0},
        {"name": "join_bwd_train", "op": "join", "dir": "bwd", "tokens": 16640, "topk": 2, "experts": 16,
         "cols": 8192, "align": 128, "dy": False, "q": True, "qt": True, "dropped": 0.0, "pad": 0},
        # The experts' gated activation: a few rows of a decoding step; the
        # forward of a training step, which keeps the two halves in 8 bits;
        # the backward from them, which also makes the activation's transposed
        # codes again for the weight gradient.
        {"name": "act_few_rows", "op": "act", "dir": "fwd", "rows": 8, "ffn": 8192, "y": False,
         "q": True, "qt": False, "save": False, "pad": 0},
        {"name": "act_train", "op": "act", "dir": "fwd", "rows": 33280, "ffn": 5120, "y": False,
         "q": True, "qt": False, "save": True, "pad": 0},
        {"name": "act_bwd_train", "op": "act", "dir": "bwd", "rows": 33280, "ffn": 5120, "codes": True,
         "dh": False, "q": True, "qt": True, "act_qt": True, "pad": 0},
        # Weight gradients of all experts: a small model's; odd sizes with
        # experts that got no token; a large layer's.
        {"name": "wgrad_small", "op": "wgrad", "experts": 8, "tokens": 2048, "m": 512, "n": 256,
         "empty": 0},
        {"name": "wgrad_odd", "op": "wgrad", "experts": 16, "tokens": 9001, "m": 1360, "n": 2064,
         "empty": 3},
        {"name": "wgrad_train", "op": "wgrad", "experts": 16, "tokens": 33280, "m": 8192, "n": 5120,
         "empty": 0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "join", "act", "wgrad"])
    if op == "wgrad":
        experts, tokens = _log(rng, 1, 64), _log(rng, 1, 33280)
        m, n = 16 * _log(rng, 4, 512), 16 * _log(rng, 4, 512)
        while experts * m * n > 16 * 8192 * 5120 or tokens * m * n > 33280 * 8192 * 5120:
            m, n = 16 * (m // 24 + 1), 16 * (n // 24 + 1)
        return {"op": op, "experts": experts, "tokens": tokens, "m": m, "n": n,
                "empty": rng.choice([0, 0, experts // 3])}
    if op == "act":
        rows, ffn = _log(rng, 1, 33280), 16 * _log(rng, 8, 640)
        while rows * ffn > 33280 * 5120:
            rows = rows // 2
        direction = rng.choice(["fwd", "bwd"])
        turned = rng.random() < 0.5
        if turned:
            rows = (rows + 15) // 16 * 16
        case = {"op": op, "dir": direction, "rows": rows, "ffn": ffn, "pad": rng.choice([0, 0, 16, 48])}
        if direction == "fwd":
            return case | {"y": not turned and rng.random() < 0.5, "q": True, "qt": turned,
                           "save": rng.random() < 0.5}
        return case | {"codes": rng.random() < 0.5, "dh": not turned, "q": turned, "qt": turned,
                       "act_qt": turned}
    tokens, topk, experts = _log(rng, 1, 16640), rng.randint(1, 8), _log(rng, 8, 256)
    cols, align = 16 * _log(rng, 8, 512), rng.choice([1, 128])
    # (an expert's padding counts as rows)
    while (tokens * topk + experts * (align - 1)) * cols > 33280 * 8192:
        tokens, experts = max(1, tokens // 2), max(8, experts * 3 // 4)
    case = {"op": op, "tokens": tokens, "topk": topk, "experts": experts, "cols": cols, "align": align,
            "dropped": rng.choice([0.0, 0.0, 0.2]), "pad": rng.choice([0, 0, 16, 48])}
    turned = align == 128 and rng.random() < 0.6
    if op == "route":
        return case | {"y": not turned and rng.random() < 0.5, "q": True, "qt": turned}
    if rng.random() < 0.5:
        return case | {"dir": "fwd", "weighted": rng.random() < 0.7}
    return case | {"dir": "bwd", "dy": not turned, "q": turned, "qt": turned}


# ---------------------------------------------------------------------------
# Inputs.

def _normal(gen, *shape, std=1.0, pad=0):
    t = torch.randn((*shape[:-1], shape[-1] + pad), generator=gen, device="cuda").mul_(std)
    return t.to(torch.bfloat16)[..., :shape[-1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = {"case": dict(case)}
    {"route": _prepare_route, "join": _prepare_join, "act": _prepare_act,
     "wgrad": _prepare_wgrad}[case["op"]](st["case"], gen, st)
    return st


def _router(case, gen):
    """A router's choice: distinct experts per token, unevenly liked, and the
    weights of the chosen ones; padding tokens go to no expert (-1)."""
    T, k, E = case["tokens"], case["topk"], case["experts"]
    logits = torch.randn(T, E, generator=gen, device="cuda")
    logits += 0.7 * torch.randn(E, generator=gen, device="cuda")
    top = torch.topk(logits, k, dim=1)
    expert = top.indices
    if case["dropped"]:
        expert = expert.masked_fill(torch.rand(T, 1, generator=gen, device="cuda") < case["dropped"], -1)
    return expert, torch.softmax(top.values, 1)


def _rows(case):
    """Rows that hold the tokens however they fall to the experts."""
    n, align = case["tokens"] * case["topk"], case["align"]
    filled = min(case["experts"], n)
    return align * (filled + (n - filled) // align)


def _prepare_route(case, gen, st):
    st["expert"], _ = _router(case, gen)
    st["x"] = _normal(gen, case["tokens"], case["cols"], pad=case["pad"])


def _prepare_join(case, gen, st):
    expert, st["weight"] = _router(case, gen)
    st["row"], st["source"], st["group_end"] = _sorted_rows(expert, case["experts"], case["align"], _rows(case))
    st["y"] = _normal(gen, _rows(case), case["cols"], pad=case["pad"])
    if case["dir"] == "bwd":
        st["dout"] = _normal(gen, case["tokens"], case["cols"], std=1e-3, pad=case["pad"])
    elif not case["weighted"]:
        st["weight"] = None


def _prepare_act(case, gen, st):
    M, F = case["rows"], case["ffn"]
    st["h"] = _normal(gen, M, 2 * F, std=1.5, pad=case["pad"])
    if case["dir"] == "bwd":
        st["dy"] = _normal(gen, M, F, std=1e-3, pad=case["pad"])
        if case["codes"]:
            st["h"], recip = _halves_1x128(st["h"].float())
            st["h_recip"] = recip.t().contiguous().t()     # column-major


def _prepare_wgrad(case, gen, st):
    E, m, n = case["experts"], case["m"], case["n"]
    share = torch.rand(E, generator=gen, device="cuda").add_(0.5)
    share[torch.randperm(E, generator=gen, device="cuda")[:case["empty"]]] = 0.0
    counts = (share / share.sum() * case["tokens"]).long().cpu()
    end = torch.cumsum((counts + 127) // 128 * 128, 0)
    # blocks behind the last expert's, where a batch filled fewer than it might have
    R = 128 * (min(E, case["tokens"]) + case["tokens"] // 128)
    st["end"] = [int(e) for e in end]
    st["group_end"] = end.to(torch.int32).cuda()
    for name, size, std in (("a", m, 1e-3), ("b", n, 1.0)):
        v = torch.randn(size, R, generator=gen, device="cuda").mul_(std)
        for e in range(E):                                 # an expert's padding rows are zero
            v[:, st["end"][e] - int((-counts[e]) % 128):st["end"][e]] = 0.0
        v = v.to(torch.bfloat16).float()
        st[name], recip = _codes_1x128(v)
        st["r" + name] = recip.t().contiguous().t()


# ---------------------------------------------------------------------------
# One pass.

def run(state):
    return {"route": _run_route, "join": _run_join, "act": _run_act,
            "wgrad": _run_wgrad}[state["case"]["op"]](state)


def _codes_1x128(v):
    """(E4M3 codes, reciprocal scales) of fp32 rows in blocks of 128 columns."""
    rows, cols = v.shape
    b = torch.nn.functional.pad(v, (0, -cols % 128)).view(rows, -1, 128)
    s = E4M3_MAX / b.abs().amax(2).clamp(min=AMAX_FLOOR)
    q = (b * s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :cols]
    return q.to(torch.float8_e4m3fn), 1.0 / s


def _halves_1x128(h):
    """The same with blocks of their own for the two halves of the columns."""
    F = h.shape[1] // 2
    q, recip = zip(_codes_1x128(h[:, :F]), _codes_1x128(h[:, F:]))
    return torch.cat([c.view(torch.uint8) for c in q], 1).view(torch.float8_e4m3fn), torch.cat(recip, 1)


def _values_1x128(q, recip):
    """fp32 values of codes in blocks of 128 columns."""
    return q.float() * recip.repeat_interleave(128, 1)[:, :q.shape[1]]


def _layouts(out, v, names):
    """v fp32 as bf16, as codes, and as codes of its transpose, under the given names (None: not)."""
    plain, q, qt = names
    if plain:
        out[plain] = v.to(torch.bfloat16)
    if q:
        out[q], out[q + "_recip"] = _codes_1x128(v)
    if qt:
        out[qt], out[qt + "_recip"] = _codes_1x128(v.t().contiguous())


def _take(out, o, **names):
    """The outputs of the package's call under the names of the plain form's."""
    for field, name in names.items():
        value = getattr(o, field)
        if value is not None:
            out[name] = value.view(torch.float8_e4m3fn) if value.dtype == torch.uint8 else value


def _sorted_rows(expert, E, align, rows):
    """(row of each slot, slot of each row, cumulative ends) of slots sorted by expert."""
    flat = expert.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    padded = (counts + align - 1) // align * align
    end = torch.cumsum(padded, 0)
    order = torch.argsort(key, stable=True)
    sorted_key = key[order]
    rank = torch.arange(n, device=flat.device) - (torch.cumsum(counts, 0) - counts)[sorted_key]
    kept = sorted_key < E
    at = torch.where(kept, (end - padded)[sorted_key] + rank, rows)
    source = torch.full((rows + 1,), -1, dtype=torch.int32, device=flat.device)
    source[at] = order.to(torch.int32)
    row = torch.empty(n, dtype=torch.int32, device=flat.device)
    row[order] = torch.where(kept, at, -1).to(torch.int32)
    return row.view(expert.shape), source[:rows], end[:E].to(torch.int32)


def _run_route(st):
    case, x = st["case"], st["x"]
    if own:
        import blockwise_scaled_fp8_amd as fp8
        table = fp8.moe_sort(st["expert"], case["experts"], align=case["align"])
        o = fp8.moe_gather(x, table, y=case["y"], q=case["q"], qt=case["qt"])
        out = {"row": table.row, "source": table.source, "group_end": table.group_end}
        _take(out, o, y="y", q="q", recip="q_recip", qt="qt", recip_t="qt_recip")
        return out
    row, source, end = _sorted_rows(st["expert"], case["experts"], case["align"], _rows(case))
    out = {"row": row, "source": source, "group_end": end}
    v = x.float()[torch.clamp(source, min=0).long() // case["topk"]]
    v = torch.where((source >= 0)[:, None], v, 0.0)
    _layouts(out, v, ("y" if case["y"] else None, "q" if case["q"] else None, "qt" if case["qt"] else None))
    return out


def _run_join(st):
    case, y, weight = st["case"], st["y"], st["weight"]
    if own:
        import blockwise_scaled_fp8_amd as fp8
        table = fp8.MoeTable(st["row"], st["source"], st["group_end"])
        if case["dir"] == "fwd":
            return {"out": fp8.moe_combine(y, table, weight)}
        o, dweight = fp8.moe_combine_bwd(st["dout"], y, table, weight, dy=case["dy"], q=case["q"], qt=case["qt"])
        out = {"dweight": dweight}
        _take(out, o, y="dy", q="q", recip="q_recip", qt="qt", recip_t="qt_recip")
        return out
    kept = st["row"] >= 0
    picked = y[torch.clamp(st["row"], min=0).long()].float()            # [T, k, H]
    picked = torch.where(kept[:, :, None], picked, 0.0)
    if case["dir"] == "fwd":
        if weight is not None:
            picked = picked * weight[:, :, None]
        return {"out": picked.sum(1).to(torch.bfloat16)}
    dout, source = st["dout"].float(), st["source"]
    out = {"dweight": (picked * dout[:, None, :]).sum(2)}
    slot = torch.clamp(source, min=0).long()
    factor = torch.where(source >= 0, weight.reshape(-1)[slot], 0.0)
    v = dout[slot // case["topk"]] * factor[:, None]
    _layouts(out, v, ("dy" if case["dy"] else None, "q" if case["q"] else None, "qt" if case["qt"] else None))
    return out


def _run_act(st):
    case, h = st["case"], st["h"]
    F = case["ffn"]
    if case["dir"] == "fwd":
        if own:
            import blockwise_scaled_fp8_amd as fp8
            o = fp8.swiglu_fwd(h, y=case["y"], q=case["q"], qt=case["qt"], save=case["save"])
            out = {}
            _take(out, o, y="y", q="q", recip="q_recip", qt="qt", recip_t="qt_recip", hq="hq", h_recip="hq_recip")
            return out
        hf = h.float()
        gate, up = hf[:, :F], hf[:, F:]
        out = {}
        _layouts(out, gate / (1.0 + torch.exp(-gate)) * up,
                 ("y" if case["y"] else None, "q" if case["q"] else None, "qt" if case["qt"] else None))
        if case["save"]:
            out["hq"], out["hq_recip"] = _halves_1x128(hf)
        return out
    if own:
        import blockwise_scaled_fp8_amd as fp8
        o = fp8.swiglu_bwd(st["dy"], h, st.get("h_recip"), dh=case["dh"], q=case["q"], qt=case["qt"],
                           act_qt=case["act_qt"])
        out = {}
        _take(out, o, dh="dh", q="q", recip="q_recip", qt="qt", recip_t="qt_recip", act_qt="act_qt",
              act_recip_t="act_qt_recip")
        return out
    if case["codes"]:
        recip, blocks = st["h_recip"], -(-F // 128)
        gate = _values_1x128(h[:, :F], recip[:, :blocks])
        up = _values_1x128(h[:, F:], recip[:, blocks:])
    else:
        gate, up = h[:, :F].float(), h[:, F:].float()
    dy = st["dy"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    silu = gate * sig
    dgate = dy * up * (sig * (1.0 + gate * (1.0 - sig)))
    dup = dy * silu
    out = {}
    dh = torch.cat([dgate, dup], 1)
    _layouts(out, dh, ("dh" if case["dh"] else None, None, "qt" if case["qt"] else None))
    if case["q"]:
        out["q"], out["q_recip"] = _halves_1x128(dh)
    if case["act_qt"]:
        _layouts(out, silu * up, (None, None, "act_qt"))
    return out


def _run_wgrad(st):
    case = st["case"]
    if own:
        import blockwise_scaled_fp8_amd as fp8
        return {"dw": fp8.fp8_scaled_grouped_gemm_blockwise_wgrad(st["a"], st["ra"], st["b"], st["rb"],
                                                                  st["group_end"])}
    dw = torch.empty(case["experts"], case["m"], case["n"], dtype=torch.bfloat16, device="cuda")
    first = 0
    for e, last in enumerate(st["end"]):                  # one expert after the other, as a plain layer
        kb = slice(first // 128, last // 128)
        dw[e] = _values_1x128(st["a"][:, first:last], st["ra"][:, kb]) @ _values_1x128(
            st["b"][:, first:last], st["rb"][:, kb]).t()
        first = last
    return {"dw": dw}


# ---------------------------------------------------------------------------
# What a pass has to move and compute.

def _layout_bytes(rows, cols, plain, q, qt):
    return (rows * cols * (2 * plain + q + qt) + 4 * rows * -(-cols // 128) * q
            + 4 * cols * -(-rows // 128) * qt)


def work(case):
    if case["op"] == "wgrad":
        # tokens, not their padding: what the gradients need
        E, T, m, n = case["experts"], case["tokens"], case["m"], case["n"]
        return {"bytes": T * (m + n) + T / 128 * 4 * (m + n) + 2 * E * m * n,
                "flops": 2 * T * m * n}
    if case["op"] == "act":
        M, F = case["rows"], case["ffn"]
        if case["dir"] == "fwd":
            moved = 4 * M * F + _layout_bytes(M, F, case["y"], case["q"], case["qt"])
            moved += 2 * M * (F + 4 * -(-F // 128)) * case["save"]
            return {"bytes": moved, "flops": 6 * M * F}
        moved = 2 * M * F + (2 * M * (F + 4 * -(-F // 128)) if case["codes"] else 4 * M * F)
        moved += _layout_bytes(M, 2 * F, case["dh"], case["q"], case["qt"])
        return {"bytes": moved + _layout_bytes(M, F, 0, 0, case["act_qt"]), "flops": 14 * M * F}
    T, n, H, R = case["tokens"], case["tokens"] * case["topk"], case["cols"], _rows(case)
    if case["op"] == "route":
        moved = 8 * n + 2 * T * H + 4 * (n + R + case["experts"])
        return {"bytes": moved + _layout_bytes(R, H, case["y"], case["q"], case["qt"]), "flops": 2 * R * H}
    if case["dir"] == "fwd":
        return {"bytes": 2 * n * H + 2 * T * H + 4 * n * (1 + case["weighted"]), "flops": 2 * n * H}
    moved = 2 * n * H + 2 * T * H + 12 * n + 4 * R
    return {"bytes": moved + _layout_bytes(R, H, case["dy"], case["q"], case["qt"]), "flops": 4 * n * H}


# ---------------------------------------------------------------------------
# The same from the definitions in 64 bits.  What is held in codes or bf16 is
# given as the value that is rounded, codes in units of their block's scale.

def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "join": _exact_join, "act": _exact_act,
            "wgrad": _exact_wgrad}[case["op"]](st)


def _exact_scaled(v):
    rows, cols = v.shape
    q, recip = torch.empty_like(v), []
    for c in range(0, cols, 128):
        block = v[:, c:c + 128]
        recip.append(block.abs().amax(1).clamp(min=AMAX_FLOOR) / E4M3_MAX)
        q[:, c:c + 128] = block / recip[-1][:, None]
    return q, torch.stack(recip, 1)


def _exact_layouts(out, v, plain, q, qt):
    if plain:
        out[plain] = v
    if q:
        out[q], out[q + "_recip"] = _exact_scaled(v)
    if qt:
        out[qt], out[qt + "_recip"] = _exact_scaled(v.t().contiguous())


def _exact_route(st):
    case, x = st["case"], st["x"].double()
    E, k, align, R = case["experts"], case["topk"], case["align"], _rows(case)
    flat = st["expert"].reshape(-1)
    row = torch.full_like(flat, -1)
    source = torch.full((R,), -1, dtype=torch.int64, device="cuda")
    v = torch.zeros(R, case["cols"], dtype=torch.float64, device="cuda")
    ends, at = [], 0
    for e in range(E):
        slots = torch.nonzero(flat == e)[:, 0]            # in order
        rows = torch.arange(at, at + len(slots), device="cuda")
        row[slots], source[rows] = rows, slots
        v[rows] = x[slots // k]
        at += -(-len(slots) // align) * align
        ends.append(at)
    out = {"row": row.view(st["expert"].shape).int(), "source": source.int(),
           "group_end": torch.tensor(ends, dtype=torch.int32, device="cuda")}
    _exact_layouts(out, v, "y" if case["y"] else None, "q" if case["q"] else None, "qt" if case["qt"] else None)
    return out


def _exact_join(st):
    case, y, row = st["case"], st["y"].double(), st["row"].long()
    T, k, H = case["tokens"], case["topk"], case["cols"]
    if case["dir"] == "fwd":
        total = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            has = torch.nonzero(row[:, j] >= 0)[:, 0]
            part = y[row[has, j]]
            total[has] += part if st["weight"] is None else part * st["weight"][has, j].double()[:, None]
        return {"out": total}
    dout = st["dout"].double()
    dweight = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    v = torch.zeros(_rows(case), H, dtype=torch.float64, device="cuda")
    for j in range(k):
        has = torch.nonzero(row[:, j] >= 0)[:, 0]
        dweight[has, j] = torch.linalg.vecdot(dout[has], y[row[has, j]])
        v[row[has, j]] = dout[has] * st["weight"][has, j].double()[:, None]
    out = {"dweight": dweight}
    _exact_layouts(out, v, "dy" if case["dy"] else None, "q" if case["q"] else None, "qt" if case["qt"] else None)
    return out


def _exact_act(st):
    case, F = st["case"], st["case"]["ffn"]
    if case["dir"] == "bwd" and case["codes"]:
        half = -(-F // 128)
        column = torch.arange(F, device="cuda") // 128
        column = torch.cat([column, half + column])
        h = st["h"].double() * st["h_recip"].double()[:, column]
    else:
        h = st["h"].double()
    gate, up = h.chunk(2, 1)
    value = torch.special.expit(gate)
    out = {}
    if case["dir"] == "fwd":
        _exact_layouts(out, gate * value * up, "y" if case["y"] else None, "q" if case["q"] else None,
                       "qt" if case["qt"] else None)
        if case["save"]:
            halves = [_exact_scaled(t.contiguous()) for t in (gate, up)]
            out["hq"], out["hq_recip"] = (torch.cat(t, 1) for t in zip(*halves))
        return out
    dy = st["dy"].double()
    slope = value + gate * value * torch.special.expit(-gate)
    dh = torch.cat([dy * up * slope, dy * gate * value], 1)
    _exact_layouts(out, dh, "dh" if case["dh"] else None, None, "qt" if case["qt"] else None)
    if case["q"]:
        halves = [_exact_scaled(t.contiguous()) for t in dh.chunk(2, 1)]
        out["q"], out["q_recip"] = (torch.cat(t, 1) for t in zip(*halves))
    if case["act_qt"]:
        _exact_layouts(out, gate * value * up, None, None, "act_qt")
    return out


def _exact_wgrad(st):
    case = st["case"]
    m, n = case["m"], case["n"]
    dw = torch.zeros(case["experts"], m, n, dtype=torch.float64, device="cuda")
    first = 0
    for e, last in enumerate(st["end"]):
        if last > first:
            a, b = (st[k][:, first:last].double().view(-1, (last - first) // 128, 128)
                    * st["r" + k][:, first // 128:last // 128].double()[:, :, None] for k in ("a", "b"))
            dw[e] = torch.mm(a.reshape(m, -1), b.reshape(n, -1).t().contiguous())
        first = last
    return {"dw": dw}
