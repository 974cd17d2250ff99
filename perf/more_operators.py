"""Cases of the router with groups and of the 8-bit block products, for timing and comparison.

    groups    routing within the best groups of experts: keys are scores plus a bias,
              top-k ids and scores, per-expert counts, the balance and z losses
    quant     E4M3 codes with one fp32 scale per 128 elements: of gathered rows, of
              SwiGLU, or of SwiGLU's gradient, along the rows and along the columns
    product   Y = X W^T on such codes, over the rows of each expert or dense
    wgrad     dW = dY^T X on codes along the columns, for each expert or dense

``own`` False: elementary torch operations in fp32 (64 bits where keys are compared),
rounded once at the end.  ``own`` True: the library's entry points.  ``exact`` gives the
same outputs from the definitions in float64.  All inputs come from the seed alone.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
BLOCK = 128
SMALLEST = 2.0 ** -100             # a block's largest magnitude counts as this at least


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one new token of a serving loop: latency is all
        {"name": "groups_token", "op": "groups", "T": 1, "E": 256, "k": 8, "groups": 8, "top": 4,
         "type": "fp32", "scoring": "sigmoid", "pair": True, "bias": True, "pad": 0, "off": 0},
        # a training step's tokens
        {"name": "groups_step", "op": "groups", "T": 8192, "E": 256, "k": 8, "groups": 8,
         "top": 4, "type": "fp32", "scoring": "sigmoid", "pair": True, "bias": True, "pad": 0,
         "off": 0},
        # a padded batch, softmax scores, many small groups, a few experts switched off
        {"name": "groups_padded", "op": "groups", "T": 16411, "E": 160, "k": 6, "groups": 20,
         "top": 5, "type": "bf16", "scoring": "softmax", "pair": False, "bias": False,
         "pad": 2048, "off": 3},
        # one token's row before a dense layer
        {"name": "quant_token", "op": "quant", "source": "rows", "M": 1, "C": 2048, "T": 1,
         "E": 1, "type": "bf16", "pow2": False, "row": True, "column": False, "clamp": 0.0},
        # a training step's rows in their experts' order, for the product and for dW
        {"name": "quant_step", "op": "quant", "source": "rows", "M": 65536, "C": 2048, "T": 8192,
         "E": 32, "type": "bf16", "pow2": False, "row": True, "column": True, "clamp": 0.0},
        # the gradient at gate and up of that step, for dX and for dW
        {"name": "quant_swiglu_grad", "op": "quant", "source": "swiglu_grad", "M": 65536,
         "C": 768, "T": 0, "E": 32, "type": "bf16", "pow2": False, "row": True, "column": True,
         "clamp": 0.0},
        # one token's experts: eight rows, each with another expert's weights
        {"name": "product_token", "op": "product", "M": 8, "N": 1536, "K": 2048, "E": 128,
         "type": "bf16", "even": False},
        # a decoding batch of 64 tokens: nearly every expert is read for a few rows
        {"name": "product_batch", "op": "product", "M": 512, "N": 1536, "K": 2048, "E": 128,
         "type": "bf16", "even": False},
        # a dense layer of odd sizes
        {"name": "product_odd", "op": "product", "M": 1003, "N": 1537, "K": 2047, "E": 1,
         "type": "fp32", "even": False},
        # the training workload's layer: 8192 tokens, 8 of 128 experts each
        {"name": "product_step", "op": "product", "M": 65536, "N": 1536, "K": 2048, "E": 128,
         "type": "bf16", "even": False},
        # a dense layer of odd sizes, weight gradient
        {"name": "wgrad_odd", "op": "wgrad", "M": 1003, "N": 777, "K": 1111, "E": 1},
        # a training step's weight gradient
        {"name": "wgrad_step", "op": "wgrad", "M": 65536, "N": 1536, "K": 2048, "E": 32},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.4 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["groups", "quant", "product", "product", "wgrad"])
    if op == "groups":
        size = rng.randint(1, 32)
        groups = rng.randint(1, 256 // size)
        top = rng.randint(1, groups)
        return {"op": op, "T": _log_int(rng, 1, 16384), "E": size * groups,
                "k": rng.randint(1, min(top * size, 16)), "groups": groups, "top": top,
                "type": rng.choice(["fp32", "bf16"]),
                "scoring": rng.choice(["sigmoid", "softmax", "softmax_topk"]),
                "pair": rng.random() < 0.5, "bias": rng.random() < 0.7,
                "pad": rng.choice([0, 1]), "off": rng.choice([0, 1])}
    E = rng.choice([1, _log_int(rng, 2, 128)])
    M = _log_int(rng, 1, 65536)
    if op == "quant":
        C = min(_width(rng, 64, 8192), 65536 * 1024 // M)
        row = rng.random() < 0.7
        source = rng.choice(["rows", "rows", "swiglu", "swiglu_grad"])
        if source != "rows":
            C = max(1, C // 2)
        return {"op": op, "source": source, "M": M, "C": C, "T": M // rng.choice([1, 8]) + 1,
                "E": E, "type": rng.choice(["bf16", "bf16", "fp32"]), "pow2": rng.random() < 0.3,
                "row": row, "column": not row or rng.random() < 0.5,
                "clamp": rng.choice([0.0, 1.5])}
    N, K = _width(rng, 64, 4096), _width(rng, 64, 4096)
    E = max(1, min(E, (1 << 28) // (N * K)))
    M = max(1, min(M, (1 << 37) // (N * K)))
    if op == "product":
        return {"op": op, "M": M, "N": N, "K": K, "E": E, "type": rng.choice(["bf16", "fp32"]),
                "even": rng.random() < 0.3}
    return {"op": op, "M": M, "N": N, "K": K, "E": E}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    op = case["op"]
    if op == "groups":
        T, E, k = case["T"], case["E"], case["k"]
        live = T - _padding(case)
        return {"bytes": live * E * (4 if case["type"] == "fp32" else 2) + T * (8 * k + 4) + 12 * E
                + 12 + (T if case["pad"] else 0), "flops": live * E * 8}
    M, E = case["M"], case["E"]
    if op == "quant":
        C, size = case["C"], 4 if case["type"] == "fp32" else 2
        read, wide = {"rows": (min(M, case["T"]) * C, C), "swiglu": (2 * M * C, C),
                      "swiglu_grad": (3 * M * C, 2 * C)}[case["source"]]
        ways = int(case["row"]) + int(case["column"])
        index = 4 * M if case["source"] == "rows" else 0
        return {"bytes": read * size + index + ways * M * (wide + 4 * _blocks(wide)),
                "flops": M * wide * 4}
    N, K = case["N"], case["K"]
    if op == "product":                # experts that some row has, expected
        seen = E * (1.0 - (1.0 - 1.0 / E) ** M) if E > 1 else 1
        return {"bytes": M * K + seen * N * K + M * N * (4 if case["type"] == "fp32" else 2)
                + 4 * M * _blocks(K), "flops": 2 * M * N * K}
    return {"bytes": M * (N + K) + 4 * E * N * K + 4 * _blocks(M) * (N + K),
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# inputs


def _padding(case):
    return case["pad"] if case["pad"] != 1 else case["T"] // 8


def _groups_inputs(case, g):
    T, E = case["T"], case["E"]
    # some experts are liked more than others, as in a trained router
    logits = torch.randn(T, E, generator=g, device=DEV) * 1.5 + torch.randn(
        E, generator=g, device=DEV) * 0.5
    bias = torch.randn(E, generator=g, device=DEV) * 0.05 if case["bias"] else None
    off = case["off"] if case["off"] != 1 else E // 8
    if off:
        logits[:, torch.randperm(E, generator=g, device=DEV)[:off]] = -math.inf
    mask = None
    if case["pad"]:
        mask = (torch.arange(T, device=DEV) < T - _padding(case)).to(torch.uint8)
    return {"logits": logits.to(TYPES[case["type"]]), "bias": bias, "mask": mask}


def _segments(M, E, g, even=False):
    """Offsets of E experts' rows (some experts are liked more than others, and a few get
    none), the first column of each when their rows are padded to whole blocks, and each
    row's expert and padded place."""
    like = torch.randn(E, generator=g, device=DEV).mul(0.0 if even else 0.5).exp()
    expert = torch.multinomial(like, M, replacement=True, generator=g).sort()[0]
    count = torch.bincount(expert, minlength=E)
    end = count.cumsum(0)
    padded = (count + BLOCK - 1) // BLOCK * BLOCK
    first = padded.cumsum(0) - padded
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    place = torch.arange(M, device=DEV) - (end - count)[expert] + first[expert]
    return {"offsets": torch.cat([zero, end]).to(torch.int32), "expert": expert, "place": place,
            "inside": torch.arange(M, device=DEV) - (end - count)[expert],
            "deepest": int(count.max()), "columns": _columns(M, E)}


def _columns(M, E):
    return _blocks(M) * BLOCK if E == 1 else (M + (BLOCK - 1) * E) // BLOCK * BLOCK


def _quant_inputs(case, g):
    M, C, dtype = case["M"], case["C"], TYPES[case["type"]]
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)
    # activations have a few channels far larger than the rest
    wide = lambda w: 1.0 + 15.0 * (torch.rand(w, generator=g, device=DEV) < 0.004)
    st = _segments(M, case["E"], g)
    if case["source"] == "rows":
        st["x"] = (n(case["T"], C) * wide(C)).to(dtype)
        rows = torch.randint(0, case["T"], (M,), generator=g, device=DEV, dtype=torch.int32)
        rows[torch.rand(M, generator=g, device=DEV) < 0.02] = -1      # padding rows
        st["rows"] = rows
        width = C
    else:
        st["a"] = n(M, 2 * C).to(dtype)
        width = C
        if case["source"] == "swiglu_grad":
            st["dh"] = (n(M, C) * 0.01).to(dtype)
            width = 2 * C
    # what the program keeps for the codes: columns that no expert has stay as they are
    ld = (width + 15) // 16 * 16
    st["by_row"] = st["by_column"] = None
    if case["row"]:
        st["by_row"] = (torch.zeros(M, ld, dtype=torch.uint8, device=DEV).view(F8)[:, :width],
                        torch.zeros(_blocks(width), M, device=DEV))
    if case["column"]:
        R = st["columns"]
        st["by_column"] = (torch.zeros(width, R, dtype=torch.uint8, device=DEV).view(F8),
                           torch.zeros(R // BLOCK, width, device=DEV))
    return st


def _codes(rows, K, g, row_blocks=None, lead=()):
    """Random codes as a quantiser leaves them: blocks scaled to the type's range, rows a
    multiple of 16 bytes apart."""
    ld = (K + 15) // 16 * 16
    v = torch.empty(*lead, rows, ld, dtype=F8, device=DEV)
    for part in v.flatten(0, -2).split(1 << 15):      # in pieces: fp32 numbers of it all are large
        part.copy_((torch.randn(part.shape, generator=g, device=DEV) * 120.0).clamp(-448, 448))
    v = v[..., :K]
    if row_blocks is None:
        s = torch.rand(*lead, _blocks(K), rows, generator=g, device=DEV)
    else:
        s = torch.rand(*lead, row_blocks, _blocks(K), generator=g, device=DEV)
    return v, (s + 0.5) / (120.0 * math.sqrt(math.sqrt(K)))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    st = {"case": case}
    if op == "groups":
        st.update(_groups_inputs(case, g))
    elif op == "quant":
        st.update(_quant_inputs(case, g))
    elif op == "product":
        M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
        st.update(_segments(M, E, g, case["even"]))
        st["x"] = _codes(M, K, g)
        st["w"] = _codes(N, K, g, _blocks(N), (E,))
    else:
        M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
        st.update(_segments(M, E, g))
        R = st["columns"]
        used = torch.zeros(R, dtype=torch.bool, device=DEV)
        used[st["place"]] = True
        for name, rows in (("dy", N), ("x", K)):       # codes of the padding are zero
            codes, scales = _codes(rows, R, g)
            codes.view(torch.uint8).mul_(used)
            st[name] = codes, scales
    if own:                        # the handle that a program keeps for the layer
        import routed_mixture_experts_gb300 as moe

        if op == "groups":
            st["handle"] = moe.MoeGroupRouter(
                case["T"], case["E"], case["k"], case["groups"], case["top"],
                dtype=TYPES[case["type"]],
                group_score=moe.MOE_GROUP_TOP2 if case["pair"] else moe.MOE_GROUP_MAX,
                scoring={"softmax_topk": moe.MOE_ROUTER_SOFTMAX_TOPK,
                         "softmax": moe.MOE_ROUTER_SOFTMAX,
                         "sigmoid": moe.MOE_ROUTER_SIGMOID}[case["scoring"]])
        elif op == "product":
            st["handle"] = moe.MoeFp8Linear(case["N"], case["K"], case["E"],
                                            dtype=TYPES[case["type"]])
        elif op == "wgrad":
            st["handle"] = moe.MoeFp8Linear(case["N"], case["K"], case["E"])
    return st


# ---------------------------------------------------------------------------
# the plain forms


def _groups(st):
    case = st["case"]
    T, E, k, scoring = case["T"], case["E"], case["k"], case["scoring"]
    G, size = case["groups"], case["E"] // case["groups"]
    l = st["logits"].float()
    live = l.amax(1) > -math.inf
    # keys in 64 bits: near ties are decided as the definition has them
    w = l.double()
    if scoring == "sigmoid":
        key = 1.0 / (1.0 + torch.exp(-w))
    else:
        key = torch.exp(w - torch.where(live, l.amax(1), 0.0)[:, None])
        key = key / key.sum(1, keepdim=True)
    if st["bias"] is not None:
        key = key + st["bias"]
    key = torch.where(l > -math.inf, key, -math.inf)
    best = key.view(T, G, size).sort(dim=2, descending=True)[0]
    value = best[:, :, 0]
    if case["pair"] and size > 1:
        value = value + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0.0)
    kept = value.sort(dim=1, descending=True, stable=True)[1][:, :case["top"]]
    stays = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter(1, kept, True)
    stays = stays.repeat_interleave(size, 1)
    # those outside the groups behind all others
    order = key.sort(dim=1, descending=True, stable=True)[1]
    inside = stays.gather(1, order).logical_not().to(torch.int8).sort(dim=1, stable=True)[1]
    ids = order.gather(1, inside)[:, :k]
    if st["mask"] is not None:     # padding tokens spread over the experts, score zero
        given = st["mask"] != 0
        live = live & given
        spread = torch.arange(T * k, device=DEV).view(T, k) % E
        ids = torch.where(given[:, None], ids, spread)
    on = live[:, None]
    c = l.gather(1, ids)
    taken = on & (c > -math.inf)
    zero = torch.zeros((), device=DEV)
    if scoring == "sigmoid":
        s = torch.where(on, 1.0 / (1.0 + torch.exp(-l)), zero)
        total = s.sum(1)
        p = torch.where(on, s / total[:, None], zero)
        stat, z = torch.log(total), torch.zeros(T, device=DEV)
        part = torch.where(taken, 1.0 / (1.0 + torch.exp(-c)), zero)
    else:
        top = torch.where(on, l.amax(1, keepdim=True), zero)
        e = torch.where(on, torch.exp(l - top), zero)
        total = e.sum(1, keepdim=True)
        p = torch.where(on, e / total, zero)
        stat = (top + torch.log(total))[:, 0]
        z = torch.where(live, stat * stat, zero)
        if scoring == "softmax":
            part = p.gather(1, ids)
        else:
            top = torch.where(taken, c, -math.inf).amax(1, keepdim=True)
            part = torch.where(taken, torch.exp(c - top), zero)
    if scoring != "softmax":
        total = part.sum(1, keepdim=True)
        part = torch.where(total > 0, part / total, zero)
    counts = torch.zeros(E + 1, device=DEV, dtype=torch.int64)
    counts.index_add_(0, ids.reshape(-1), taken.reshape(-1).long())
    n = live.sum()
    counts[E] = n
    prob_sum = p.sum(0)
    nf = n.float().clamp(min=1.0)
    balance = (counts[:E].float() * prob_sum).sum() * (E / k) / (nf * nf)
    return {"ids": ids.to(torch.int32), "scores": torch.where(taken, part, zero),
            "counts": counts.to(torch.int32), "prob_sum": prob_sum,
            "losses": torch.stack([balance, z.sum() / nf]), "row_stat": stat}


def _source(st):
    case = st["case"]
    if case["source"] == "rows":
        v = st["x"].float()[st["rows"].long().clamp(min=0)]
        return torch.where(st["rows"][:, None] >= 0, v, 0.0)
    C, limit = case["C"], case["clamp"]
    a = st["a"].float()
    gate, up = a[:, :C], a[:, C:]
    within_gate = within_up = 1.0
    if limit:
        within_gate, within_up = gate.abs() <= limit, up.abs() <= limit
        gate, up = gate.clamp(-limit, limit), up.clamp(-limit, limit)
    s = 1.0 / (1.0 + torch.exp(-gate))
    if case["source"] == "swiglu":
        return gate * s * up
    dh = st["dh"].float()
    d_gate = dh * up * s * (1.0 + gate * (1.0 - s)) * within_gate
    return torch.cat([d_gate, dh * gate * s * within_up], 1)


def _block_codes(v, pow2):
    """[rows, K], K whole blocks -> codes and scales [K / 128, rows]."""
    b = v.view(v.shape[0], -1, BLOCK)
    top = b.abs().amax(2).clamp(min=SMALLEST)
    if pow2:
        m, e = torch.frexp(top / 448.0)           # the power of two at or above
        e = torch.where(m == 0.5, e - 1, e)
        scale, inverse = ((127 + i << 23).view(torch.float32) for i in (e, -e))
    else:
        scale, inverse = top / 448.0, 448.0 / top
    return (b * inverse[:, :, None]).to(F8).view(v.shape), scale.t().contiguous()


def _quant(st):
    case = st["case"]
    v = _source(st)
    M, width = v.shape
    out = {}
    if case["row"]:
        wide = torch.zeros(M, _blocks(width) * BLOCK, device=DEV)
        wide[:, :width] = v
        codes, scales = _block_codes(wide, case["pow2"])
        out["codes"], out["scales"] = codes[:, :width], scales
    if case["column"]:
        R = st["columns"]
        tall = torch.zeros(width, R, device=DEV)
        tall[:, st["place"]] = v.t()
        codes, scales = _block_codes(tall, case["pow2"])
        used = torch.zeros(R // BLOCK, dtype=torch.bool, device=DEV)
        used[st["place"] // BLOCK] = True
        out["codes_t"], out["scales_t"] = codes, torch.where(used[:, None], scales, 0.0)
    return out


def _values(codes, scales, dtype=torch.float32):
    """[rows, K] of row codes."""
    K = codes.shape[1]
    return codes.to(dtype) * scales.to(dtype).t().repeat_interleave(BLOCK, 1)[:, :K]


def _weights(codes, scales, dtype=torch.float32):
    N, K = codes.shape[-2:]
    s = scales.to(dtype).repeat_interleave(BLOCK, -2)[..., :N, :]
    return codes.to(dtype) * s.repeat_interleave(BLOCK, -1)[..., :K]


def _product(st):
    case = st["case"]
    M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
    x = _values(*st["x"])
    if E == 1:
        y = x @ _weights(*st["w"])[0].t()
    elif M < E:                        # few rows: each with its own expert's weights
        w = _weights(st["w"][0][st["expert"]], st["w"][1][st["expert"]])
        y = torch.bmm(w, x[:, :, None])[:, :, 0]
    else:                              # every expert with as many rows as the busiest has
        padded = torch.zeros(E, st["deepest"], K, device=DEV)
        padded[st["expert"], st["inside"]] = x
        y = torch.bmm(padded, _weights(*st["w"]).transpose(1, 2))[st["expert"], st["inside"]]
    return y.to(TYPES[case["type"]])


def _wgrad(st):
    case = st["case"]
    M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
    dy, x = _values(*st["dy"]).t()[st["place"]], _values(*st["x"]).t()[st["place"]]
    if E == 1:
        return (dy.t() @ x)[None]
    a = torch.zeros(E, st["deepest"], N, device=DEV)
    b = torch.zeros(E, st["deepest"], K, device=DEV)
    a[st["expert"], st["inside"]] = dy
    b[st["expert"], st["inside"]] = x
    return torch.bmm(a.transpose(1, 2), b)


# ---------------------------------------------------------------------------
# one pass


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"groups": _groups, "quant": _quant, "product": _product, "wgrad": _wgrad}[op](st)
    import routed_mixture_experts_gb300 as moe

    if op == "groups":
        r = st["handle"].forward(st["logits"], bias=st["bias"], token_mask=st["mask"])
        return {"ids": r.ids, "scores": r.scores, "counts": r.counts, "prob_sum": r.prob_sum,
                "losses": r.losses, "row_stat": r.row_stat}
    offsets = st["offsets"] if case["E"] > 1 else None
    if op == "quant":
        out = dict(offsets=offsets, pow2=case["pow2"], by_row=case["row"],
                   by_column=case["column"], out=st["by_row"], out_t=st["by_column"])
        if case["source"] == "rows":
            q, t = moe.quantize_fp8(st["x"], rows=st["rows"], **out)
        elif case["source"] == "swiglu":
            q, t = moe.swiglu_fp8(st["a"], clamp=case["clamp"], **out)
        else:
            q, t = moe.swiglu_grad_fp8(st["dh"], st["a"], clamp=case["clamp"], **out)
        res = {}
        if q is not None:
            res["codes"], res["scales"] = q
        if t is not None:
            res["codes_t"], res["scales_t"] = t
        return res
    if op == "product":
        return st["handle"].forward(st["x"], st["w"], offsets=offsets)
    return st["handle"].grad_weight(st["dy"], st["x"], offsets=offsets)


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_choice(key, T, E, k, G, top, pair):
    """ids by counting those ahead, ties to the lowest index."""
    size = E // G
    first = torch.ones(E, E, dtype=torch.bool, device=DEV).tril(-1)     # [e, i]: i < e
    ids = torch.empty(T, k, dtype=torch.int64, device=DEV)
    for t in range(0, T, 1024):
        a = key[t:t + 1024]
        n = a.shape[0]
        b = a.view(n, G, size).topk(min(2, size), dim=2)[0]
        v = b[:, :, 0].clone()
        if pair and size > 1:
            v += torch.where(b[:, :, 1] == -math.inf, torch.zeros_like(v), b[:, :, 1])
        f = first[:G, :G]
        ahead = ((v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & f)).sum(2)
        stays = (ahead < top).repeat_interleave(size, 1)
        better = (a[:, None, :] > a[:, :, None]) | ((a[:, None, :] == a[:, :, None]) & first)
        place = (better & stays[:, None, :]).sum(2)
        place = torch.where(stays, place, E + torch.arange(E, device=DEV))
        ids[t:t + 1024] = place.argsort(1)[:, :k]
    return ids


def _exact_groups(st):
    case = st["case"]
    T, E, k, scoring = case["T"], case["E"], case["k"], case["scoring"]
    l = st["logits"].double()
    live = torch.isfinite(l).any(1)
    p = torch.sigmoid(l) if scoring == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    key = p if st["bias"] is None else p + st["bias"].double()
    key = torch.where(l == -math.inf, -math.inf, key)
    ids = _exact_choice(key, T, E, k, case["groups"], case["top"], case["pair"])
    if st["mask"] is not None:
        live &= st["mask"].bool()
    n = live.double().sum().clamp(min=1)
    chosen = l.gather(1, ids)
    hit = live[:, None] & (chosen > -math.inf)
    if scoring == "softmax":
        s = p.gather(1, ids)
    elif scoring == "sigmoid":
        s = torch.sigmoid(chosen)
        s = s / s.sum(1, keepdim=True)
    else:
        s = torch.softmax(chosen, 1)
    if scoring == "sigmoid":
        total = p.sum(1)
        p, stat = p / total[:, None], total.log()
        z = 0.0 * n
    else:
        stat = torch.logsumexp(l, 1)
        z = stat[live].square().sum() / n
    p = torch.where(live[:, None], p, 0.0)
    counts = torch.bincount(ids[hit], minlength=E).double()
    balance = E * ((counts / (k * n)) * (p.sum(0) / n)).sum()
    return {"ids": None, "scores": torch.where(hit, s, 0.0), "counts": None, "prob_sum": p.sum(0),
            "losses": torch.stack([balance, z]), "row_stat": torch.where(live, stat, -math.inf)}


def _exact_quant(st):
    """Codes as the quotients that they round."""
    case = st["case"]
    C, limit = case["C"], case["clamp"]
    if case["source"] == "rows":
        v = torch.cat([st["x"].double(), torch.zeros(1, C, dtype=torch.float64, device=DEV)])
        v = v[st["rows"].long()]                       # -1: the row of zeros
    else:
        with torch.enable_grad():
            a = st["a"].double().requires_grad_(True)
            c = a.clamp(-limit, limit) if limit else a
            h = torch.nn.functional.silu(c[:, :C]) * c[:, C:]
            v = h.detach()
            if case["source"] == "swiglu_grad":
                (v,) = torch.autograd.grad(h, a, st["dh"].double())

    def codes(m):
        rows, K = m.shape
        parts = [m[:, k:k + BLOCK] for k in range(0, K, BLOCK)]
        top = torch.stack([q.abs().amax(1) for q in parts]).clamp(min=SMALLEST)
        scale = top / 448.0
        if case["pow2"]:
            scale = torch.exp2(torch.ceil(torch.log2(scale) - 1e-12))
        return torch.cat([q / s[:, None] for q, s in zip(parts, scale)], 1), scale

    out = {}
    if case["row"]:
        out["codes"], out["scales"] = codes(v)
    if case["column"]:
        tall = torch.zeros(st["columns"], v.shape[1], dtype=torch.float64, device=DEV)
        tall[st["place"]] = v
        q, s = codes(tall.t())
        used = torch.zeros(st["columns"] // BLOCK, 1, dtype=torch.bool, device=DEV)
        used[st["place"] // BLOCK] = True
        out["codes_t"], out["scales_t"] = q, torch.where(used, s, 0.0)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "groups":
        return _exact_groups(st)
    if op == "quant":
        return _exact_quant(st)
    M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
    if M * N * K > 1 << 38:            # 64-bit products of it would take too long
        return None
    ends = st["offsets"].tolist()

    def scaled(codes, scales, lo, hi):
        """Columns lo to hi of row codes."""
        v = codes[:, lo:hi].double()
        for b in range(lo // BLOCK, (hi + BLOCK - 1) // BLOCK):
            v[:, max(b * BLOCK - lo, 0):(b + 1) * BLOCK - lo] *= scales[b].double()[:, None]
        return v

    if op == "product":
        y = torch.zeros(M, N, dtype=torch.float64, device=DEV)
        for e in range(E):
            if ends[e + 1] > ends[e]:
                codes, scales = st["w"][0][e].double(), st["w"][1][e].double()
                for n in range(0, N, BLOCK):
                    codes[n:n + BLOCK] *= scales[n // BLOCK].repeat_interleave(BLOCK)[:K]
                rows = slice(ends[e], ends[e + 1])
                y[rows] = scaled(st["x"][0][rows], st["x"][1][:, rows], 0, K) @ codes.t()
        return y
    dw = torch.zeros(E, N, K, dtype=torch.float64, device=DEV)
    at = 0
    for e in range(E):
        n = ends[e + 1] - ends[e]
        if n:
            dw[e] = scaled(*st["dy"], at, at + n) @ scaled(*st["x"], at, at + n).t()
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    return dw
