"""Cases of the operators around the routed experts, for timing and comparison.

    route, route_grad   the router: top-k ids and scores from logits, per-expert
                        counts, the balance and z losses; its gradient
    norm, norm_grad     the norm after a block with its gate and residual scale,
                        joined with the norm before the next one; its gradient
    decode              the routed experts of a few tokens on 4-bit weights
                        (E2M1 codes, E4M3 scales per 16, one fp32 scale per expert)

``own`` False: elementary torch operations in fp32, rounded once at the end.
``own`` True: the library's entry points.  ``exact`` gives the same outputs from
the definitions in float64.  All inputs come from the seed alone.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one new token of a serving loop: latency is all
        {"name": "route_token", "op": "route", "T": 1, "E": 128, "k": 8, "type": "fp32",
         "scoring": "softmax_topk", "bias": False, "pad": 0, "off": 0},
        # the training workload's layer (T=8192, E=128, k=8)
        {"name": "route_step", "op": "route", "T": 8192, "E": 128, "k": 8, "type": "fp32",
         "scoring": "softmax_topk", "bias": False, "pad": 0, "off": 0},
        # a padded batch on a router with a selection bias, a few experts switched off
        {"name": "route_padded", "op": "route", "T": 16411, "E": 250, "k": 6, "type": "bf16",
         "scoring": "sigmoid", "bias": True, "pad": 2048, "off": 3},
        # the training workload's layer, backward
        {"name": "route_grad_step", "op": "route_grad", "T": 8192, "E": 128, "k": 8,
         "type": "fp32", "scoring": "softmax_topk", "bias": False, "pad": 0, "off": 0},
        # the padded batch, backward
        {"name": "route_grad_padded", "op": "route_grad", "T": 16411, "E": 250, "k": 6,
         "type": "bf16", "scoring": "sigmoid", "bias": True, "pad": 2048, "off": 3},
        # one new token between two blocks
        {"name": "norm_token", "op": "norm", "T": 1, "d": 2048, "act": "bf16", "res": "bf16",
         "gate": "channel", "alpha": 1.0},
        # the training workload's layer (T=8192, d=2048)
        {"name": "norm_step", "op": "norm", "T": 8192, "d": 2048, "act": "bf16", "res": "bf16",
         "gate": "channel", "alpha": 0.5},
        # the training workload's layer, backward
        {"name": "norm_grad_step", "op": "norm_grad", "T": 8192, "d": 2048, "act": "bf16",
         "res": "bf16", "gate": "channel", "alpha": 0.5},
        # an odd width and length with an fp32 residual stream and a gate for each token
        {"name": "norm_grad_odd", "op": "norm_grad", "T": 4099, "d": 1537, "act": "bf16",
         "res": "fp32", "gate": "token", "alpha": 1.0},
        # one sequence's next token on the training workload's layer
        {"name": "decode_token", "op": "decode", "T": 1, "d": 2048, "I": 768, "E": 128, "k": 8},
        # a handful of sequences on few experts, so that experts share tokens
        {"name": "decode_few", "op": "decode", "T": 7, "d": 2048, "I": 768, "E": 16, "k": 8},
        # a full decoding batch: every expert is read
        {"name": "decode_batch", "op": "decode", "T": 64, "d": 2048, "I": 768, "E": 128, "k": 8},
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["route", "route_grad", "norm", "norm_grad", "decode"])
    if op in ("route", "route_grad"):
        E = _log_int(rng, 4, 256)
        T = _log_int(rng, 1, 16384)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 16)),
                "type": rng.choice(["fp32", "bf16"]),
                "scoring": rng.choice(["softmax_topk", "softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "pad": rng.choice([0, T // 8]),
                "off": rng.choice([0, E // 8])}
    if op in ("norm", "norm_grad"):
        T = _log_int(rng, 1, 8192)
        act = rng.choice(["bf16", "bf16", "fp32"])
        d = min(_log_int(rng, 64, 8192), 8192 * (1024 if act == "fp32" else 2048) // T)
        d = d if rng.random() < 0.4 else max(64, d // 64 * 64)
        return {"op": op, "T": T, "d": d + 64 if d == 3072 else d, "act": act,
                "res": "fp32" if act == "fp32" else rng.choice(["bf16", "fp32"]),
                "gate": rng.choice(["none", "channel", "token"]),
                "alpha": rng.choice([1.0, 0.25])}
    E = _log_int(rng, 4, 128)
    return {"op": op, "T": _log_int(rng, 1, 64), "d": rng.choice([256, 512, 1024, 1280, 2048]),
            "I": rng.choice([256, 512, 768]), "E": E, "k": rng.randint(1, min(E, 8))}


def work(case):
    op, T = case["op"], case["T"]
    if op in ("route", "route_grad"):
        E, k = case["E"], case["k"]
        size = 4 if case["type"] == "fp32" else 2
        live = T - case["pad"]
        if op == "route":
            # logits in; ids, scores, one statistic a token out; counts, sums and losses
            return {"bytes": live * E * size + T * (8 * k + 4) + 8 * E + 16
                    + (4 * E if case["bias"] else 0) + (T if case["pad"] else 0),
                    "flops": live * E * 6}
        return {"bytes": live * E * size + T * E * size + T * (8 * k + 4) + 4 * E,
                "flops": live * E * 8}
    if op in ("norm", "norm_grad"):
        d = case["d"]
        a, r = (4 if case[n] == "fp32" else 2 for n in ("act", "res"))
        gate = {"none": 0, "channel": 4 * d, "token": 4 * T}[case["gate"]]
        if op == "norm":   # residual, y in; residual, u out; two weights
            return {"bytes": T * d * (2 * a + 2 * r) + 8 * d + gate, "flops": T * d * 9}
        # residual, its gradient, y, du in; dresidual, dy out; weights and their gradients
        return {"bytes": T * d * (3 * r + 3 * a) + 16 * d + 2 * gate, "flops": T * d * 24}
    d, I, E, k = case["d"], case["I"], case["E"], case["k"]
    read = E * (1.0 - (1.0 - k / E) ** T)        # experts that some token chose, expected
    per = 3 * d * I / 2 * (1 + 1 / 8) + 8        # codes, a scale byte per 16, two scales
    return {"bytes": read * per + T * (4 * d + 8 * k), "flops": T * k * 6 * d * I}


# ---------------------------------------------------------------------------
# inputs


def _route_inputs(case, g):
    T, E, k = case["T"], case["E"], case["k"]
    # some experts are liked more than others, as in a trained router
    logits = torch.randn(T, E, generator=g, device=DEV) * 1.5 + torch.randn(
        E, generator=g, device=DEV) * 0.5
    bias = torch.randn(E, generator=g, device=DEV) * 0.2 if case["bias"] else None
    if case["off"]:
        gone = torch.randperm(E, generator=g, device=DEV)[: case["off"]]
        logits[:, gone] = -math.inf
    logits = logits.to(TYPES[case["type"]])
    mask = None
    if case["pad"]:
        mask = (torch.arange(T, device=DEV) < T - case["pad"]).to(torch.uint8)
    return {"logits": logits, "bias": bias, "mask": mask}


def _norm_inputs(case, g):
    T, d = case["T"], case["d"]
    act, res = TYPES[case["act"]], TYPES[case["res"]]
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)
    # a residual stream has a few channels far larger than the rest
    wide = 1.0 + 15.0 * (torch.rand(d, generator=g, device=DEV) < 0.004)
    st = {"residual": (n(T, d) * wide).to(res), "y": (n(T, d) * 0.3).to(act),
          "w_post": 1.0 + 0.1 * n(d), "w_pre": 1.0 + 0.1 * n(d), "gate": None}
    if case["gate"] == "channel":
        st["gate"] = 0.5 + 0.2 * n(d)
    elif case["gate"] == "token":
        st["gate"] = torch.rand(T, generator=g, device=DEV)
    if case["op"] == "norm_grad":
        st["d_residual"] = (n(T, d) * 0.01).to(res)
        st["d_u"] = (n(T, d) * 0.01).to(act)
    return st


def _decode_inputs(case, g):
    T, d, I, E, k = (case[n] for n in ("T", "d", "I", "E", "k"))
    code = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.uint8)
    # E4M3 scale codes of 16 up to 448: blocks of a tensor scaled to the type's range
    scale = lambda n: torch.randint(0x58, 0x7F, (n,), generator=g, device=DEV, dtype=torch.uint8)
    spread = lambda K: (0.5 + torch.rand(E, generator=g, device=DEV)) / (600.0 * math.sqrt(K))
    return {
        "x": torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16),
        "ids": torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].to(
            torch.int32).contiguous(),
        "scores": torch.randn(T, k, generator=g, device=DEV).softmax(1),
        # codes [E, 2I, d/2], [E, d, I/2] and the tiled scales of prepared weights
        "w13": (code(E, 2 * I, d // 2), scale(E * 2 * I * d // 16), spread(d)),
        "w2": (code(E, d, I // 2), scale(E * d * I // 16), spread(I)),
    }


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    st = {"case": case}
    if op in ("route", "route_grad"):
        st.update(_route_inputs(case, g))
        if op == "route_grad":     # what the forward left, and the gradients that arrive
            f = _route(st)
            st.update(ids=f["ids"], counts=f["counts"], row_stat=f["row_stat"])
            st["d_scores"] = torch.randn(case["T"], case["k"], generator=g, device=DEV) * 0.01
            st["d_losses"] = torch.tensor(
                [0.01, 0.0 if case["scoring"] == "sigmoid" else 0.001], device=DEV)
    elif op in ("norm", "norm_grad"):
        st.update(_norm_inputs(case, g))
    else:
        st.update(_decode_inputs(case, g))
    if own:                        # the handle that a program keeps for the layer
        import routed_mixture_experts_gb300 as moe

        if op in ("route", "route_grad"):
            st["handle"] = moe.MoeRouter(
                case["T"], case["E"], case["k"], dtype=TYPES[case["type"]],
                scoring={"softmax_topk": moe.MOE_ROUTER_SOFTMAX_TOPK,
                         "softmax": moe.MOE_ROUTER_SOFTMAX,
                         "sigmoid": moe.MOE_ROUTER_SIGMOID}[case["scoring"]])
        elif op in ("norm", "norm_grad"):
            st["handle"] = moe.MoeBlockNorm(
                case["T"], case["d"], dtype=TYPES[case["act"]],
                residual_dtype=TYPES[case["res"]], alpha=case["alpha"], eps=EPS,
                gate={"none": moe.MOE_GATE_NONE, "channel": moe.MOE_GATE_CHANNEL,
                      "token": moe.MOE_GATE_TOKEN}[case["gate"]])
        else:
            st["handle"] = moe.MoePlan(case["T"], case["d"], case["I"], case["E"], case["k"],
                                       precision=moe.MOE_PREC_NVFP4, flags=0)
    return st


# ---------------------------------------------------------------------------
# the plain forms (fp32, rounded once at the end)


def _chosen(values, ids):
    return values.gather(1, ids.long())


def _route(st):
    case = st["case"]
    T, E, k, scoring = case["T"], case["E"], case["k"], case["scoring"]
    l = st["logits"].float()
    live = l.amax(1) > -math.inf
    key = l if st["bias"] is None else l + st["bias"]
    ids = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
    if st["mask"] is not None:     # padding tokens spread over the experts, score zero
        given = st["mask"] != 0
        live = live & given
        spread = torch.arange(T * k, device=DEV).view(T, k) % E
        ids = torch.where(given[:, None], ids, spread)
    on = live[:, None]
    c = _chosen(l, ids)
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
            part = _chosen(p, ids)
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
    return {"ids": ids.to(torch.int32), "scores": torch.where(on, part, zero),
            "counts": counts.to(torch.int32), "prob_sum": prob_sum,
            "losses": torch.stack([balance, z.sum() / nf]), "row_stat": stat}


def _route_grad(st):
    case = st["case"]
    E, k, scoring = case["E"], case["k"], case["scoring"]
    l = st["logits"].float()
    stat = st["row_stat"][:, None]
    on = stat > -math.inf
    zero = torch.zeros((), device=DEV)
    nf = st["counts"][E].float().clamp(min=1.0)
    gp = st["d_losses"][0] * (E / k) * st["counts"][:E].float() / (nf * nf)
    c = _chosen(l, st["ids"])
    taken = on & (c > -math.inf)
    ds = torch.where(taken, st["d_scores"], zero)
    if scoring == "sigmoid":
        s = torch.where(on, 1.0 / (1.0 + torch.exp(-l)), zero)
        total = torch.exp(stat)
        p = torch.where(on, s / total, zero)
        gs = torch.where(on, (gp - (gp * p).sum(1, keepdim=True)) / total, zero)
        part = torch.where(taken, 1.0 / (1.0 + torch.exp(-c)), zero)
        total = part.sum(1, keepdim=True)
        part = torch.where(total > 0, part / total, zero)
        mean = (ds * part).sum(1, keepdim=True)
        gc = torch.where(taken & (total > 0), (ds - mean) / total, zero)
        gs = gs.expand_as(l).scatter_add(1, st["ids"].long(), gc)
        return torch.where(on, gs * s * (1.0 - s), zero).to(st["logits"].dtype)
    p = torch.where(on, torch.exp(l - stat), zero)
    g = gp.expand_as(l)
    if scoring == "softmax":
        g = g.scatter_add(1, st["ids"].long(), ds)
    dl = p * (g - (g * p).sum(1, keepdim=True))
    dl = dl + p * torch.where(on, st["d_losses"][1] * 2.0 * stat / nf, zero)
    if scoring == "softmax_topk":
        top = torch.where(taken, c, -math.inf).amax(1, keepdim=True)
        part = torch.where(taken, torch.exp(c - top), zero)
        total = part.sum(1, keepdim=True)
        part = torch.where(total > 0, part / total, zero)
        dl = dl.scatter_add(1, st["ids"].long(), part * (ds - (ds * part).sum(1, keepdim=True)))
    return torch.where(on, dl, zero).to(st["logits"].dtype)


def _inverse_rms(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def _gate(st):
    if st["gate"] is None:
        return 1.0
    return st["gate"][:, None] if st["case"]["gate"] == "token" else st["gate"]


def _norm(st):
    y, r = st["y"].float(), st["residual"].float()
    out = r + st["case"]["alpha"] * _gate(st) * (y * _inverse_rms(y) * st["w_post"])
    u = out * _inverse_rms(out) * st["w_pre"]
    return out.to(st["residual"].dtype), u.to(st["y"].dtype)


def _norm_grad(st):
    case = st["case"]
    r, y, du = st["residual"].float(), st["y"].float(), st["d_u"].float()
    scale = _inverse_rms(r)
    rhat = r * scale
    t = du * st["w_pre"]
    dr = st["d_residual"].float() + scale * (t - rhat * (t * rhat).mean(1, keepdim=True))
    scale = _inverse_rms(y)
    yhat = y * scale
    dn = case["alpha"] * _gate(st) * dr
    t = dn * st["w_post"]
    dy = scale * (t - yhat * (t * yhat).mean(1, keepdim=True))
    out = {"d_residual": dr.to(st["residual"].dtype), "dy": dy.to(st["y"].dtype),
           "dw_pre": (du * rhat).sum(0), "dw_post": (dn * yhat).sum(0)}
    if st["gate"] is not None:
        out["dgate"] = (case["alpha"] * dr * yhat * st["w_post"]).sum(
            1 if case["gate"] == "token" else 0)
    return out


def _scale_offsets(rows, K, gate_up):
    """Byte of the tiled scales for row r and 16-element block b of one expert."""
    r = torch.arange(rows, device=DEV)
    if gate_up:                    # 64 gate rows, then the same 64 up rows
        half = rows // 2
        up = (r >= half).long()
        i = r - up * half
        block, r = i // 64, up * 64 + i % 64
    else:
        block, r = r // 128, r % 128
    b = torch.arange(K // 16, device=DEV)
    at = (block[:, None] * (K // 64) + b // 4) * 512
    return at + ((r % 32) * 16 + r // 32 * 4)[:, None] + b % 4


def _dequantise(weights, experts, K, gate_up):
    codes, scales, whole = weights
    E, rows = codes.shape[:2]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    c = codes[experts]
    v = table[torch.stack([c & 15, c >> 4], -1).int()].view(-1, rows, K // 16, 16)
    s = scales.view(E, -1)[experts][:, _scale_offsets(rows, K, gate_up)]
    v = v * s.view(torch.float8_e4m3fn).float()[..., None]
    return (v * whole[experts].view(-1, 1, 1, 1)).view(-1, rows, K)


def _decode(st):
    case = st["case"]
    T, d, I, E, k = (case[n] for n in ("T", "d", "I", "E", "k"))
    x, ids = st["x"].float(), st["ids"].long()
    if T * k < E:                  # each token with each of its experts
        experts = ids.reshape(-1)
        xs = x.repeat_interleave(k, 0)[:, :, None]
    else:                          # every expert with every token
        experts = torch.arange(E, device=DEV)
        xs = x.t().expand(E, d, T)
    a = torch.bmm(_dequantise(st["w13"], experts, d, True), xs)
    gate, up = a[:, :I], a[:, I:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    o = torch.bmm(_dequantise(st["w2"], experts, I, False), h)
    if T * k < E:
        y = (o.view(T, k, d) * st["scores"][:, :, None]).sum(1)
    else:
        weight = torch.zeros(T, E, device=DEV).scatter_add(1, ids, st["scores"])
        y = torch.einsum("edt,te->td", o, weight)
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# one pass


def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        return {"route": _route, "route_grad": _route_grad, "norm": _norm,
                "norm_grad": _norm_grad, "decode": _decode}[op](st)
    h = st["handle"]
    if op == "route":
        r = h.forward(st["logits"], bias=st["bias"], token_mask=st["mask"])
        return {"ids": r.ids, "scores": r.scores, "counts": r.counts, "prob_sum": r.prob_sum,
                "losses": r.losses, "row_stat": r.row_stat}
    if op == "route_grad":
        return h.backward(st["logits"], st["ids"], st["counts"], st["row_stat"],
                          d_scores=st["d_scores"], d_losses=st["d_losses"])
    if op == "norm":
        return h.forward(st["residual"], y=st["y"], w_post=st["w_post"], gate=st["gate"],
                         w_pre=st["w_pre"])
    if op == "norm_grad":
        r = h.backward(st["residual"], st["d_residual"], st["d_u"], y=st["y"],
                       w_post=st["w_post"], gate=st["gate"], w_pre=st["w_pre"])
        out = {"d_residual": r.d_residual, "dy": r.dy, "dw_pre": r.dw_pre, "dw_post": r.dw_post}
        if r.dgate is not None:
            out["dgate"] = r.dgate
        return out
    return h.decode_nvfp4(st["x"], st["ids"], st["scores"], st["w13"] + st["w2"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_choice(key, k):
    """The k largest of each row by counting those ahead, ties to the lowest index."""
    T, E = key.shape
    first = torch.ones(E, E, dtype=torch.bool, device=DEV).tril(-1)     # [e, i]: i < e
    out = torch.empty(T, k, dtype=torch.int64, device=DEV)
    for t in range(0, T, 1024):
        a = key[t:t + 1024]
        ahead = (a[:, None, :] > a[:, :, None]) | ((a[:, None, :] == a[:, :, None]) & first)
        place = ahead.sum(2)
        out[t:t + 1024] = place.argsort(1)[:, :k]
    return out


def _exact_probabilities(l, live, scoring):
    """(p, statistic) of each live row; zeros elsewhere."""
    if scoring == "sigmoid":
        s = torch.sigmoid(l)
        total = s.sum(1)
        p, stat = s / total[:, None], torch.where(live, total.log(), -math.inf)
    else:
        stat = torch.logsumexp(l, 1)
        p, stat = torch.softmax(l, 1), torch.where(live, stat, -math.inf)
    return torch.where(live[:, None], p, 0.0), stat


def _exact_scores(l, ids, live, scoring):
    c = l.gather(1, ids)
    if scoring == "softmax":
        s = torch.softmax(l, 1).gather(1, ids)
    elif scoring == "sigmoid":
        s = torch.sigmoid(c)
        s = s / s.sum(1, keepdim=True)
    else:
        s = torch.softmax(c, 1)
    return torch.where(live[:, None], torch.nan_to_num(s), 0.0)


def _exact_losses(counts, p, stat, live, n, E, k, scoring):
    balance = E * ((counts / (k * n)) * (p.sum(0) / n)).sum()
    z = 0.0 * n if scoring == "sigmoid" else stat[live].square().sum() / n
    return torch.stack([balance, z])


def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op in ("route", "route_grad"):
        E, k, scoring = case["E"], case["k"], case["scoring"]
        l = st["logits"].double()
        live = torch.isfinite(l).any(1)
        if st["mask"] is not None:
            live &= st["mask"].bool()
        n = live.double().sum().clamp(min=1)
        if op == "route":
            key = st["logits"].float()
            ids = _exact_choice(key if st["bias"] is None else key + st["bias"], k)
            p, stat = _exact_probabilities(l, live, scoring)
            hit = live[:, None] & (l.gather(1, ids) > -math.inf)
            counts = torch.bincount(ids[hit], minlength=E).double()
            return {"ids": None, "scores": _exact_scores(l, ids, live, scoring), "counts": None,
                    "prob_sum": p.sum(0), "row_stat": stat,
                    "losses": _exact_losses(counts, p, stat, live, n, E, k, scoring)}
        # differentiate the forward's definition
        with torch.enable_grad():
            rows = l[live].requires_grad_(True)
            every = torch.ones(rows.shape[0], dtype=torch.bool, device=DEV)
            ids = st["ids"].long()[live]
            p, stat = _exact_probabilities(rows, every, scoring)
            counts = st["counts"][:E].double()
            losses = _exact_losses(counts, p, stat, every, n, E, k, scoring)
            s = _exact_scores(rows, ids, every, scoring)
            total = (s * st["d_scores"].double()[live]).sum() + (
                losses * st["d_losses"].double()).sum()
            (grad,) = torch.autograd.grad(total, rows)
        out = torch.zeros_like(l)
        out[live] = torch.nan_to_num(grad)
        return out
    if op in ("norm", "norm_grad"):
        names = ["residual", "y", "w_post", "w_pre"] + (["gate"] if st["gate"] is not None else [])
        v = {n: st[n].double().requires_grad_(op == "norm_grad") for n in names}
        with torch.set_grad_enabled(op == "norm_grad"):
            y = v["y"]
            n = y / (y.square().sum(1, keepdim=True) / case["d"] + EPS).sqrt() * v["w_post"]
            if "gate" in v:
                n = n * (v["gate"].view(T, 1) if case["gate"] == "token" else v["gate"])
            move = case["alpha"] * n
            # the backward's residual is the stream after the block
            out = v["residual"] + (move if op == "norm" else move - move.detach())
            u = out / (out.square().sum(1, keepdim=True) / case["d"] + EPS).sqrt() * v["w_pre"]
            if op == "norm":
                return out, u
            total = (out * st["d_residual"].double()).sum() + (u * st["d_u"].double()).sum()
            got = dict(zip(names, torch.autograd.grad(total, [v[n] for n in names])))
        res = {"d_residual": got["residual"], "dy": got["y"], "dw_pre": got["w_pre"],
               "dw_post": got["w_post"]}
        if "gate" in v:
            res["dgate"] = got["gate"]
        return res
    d, I, E, k = (case[n] for n in ("d", "I", "E", "k"))
    x, ids = st["x"].double(), st["ids"].long()
    y = torch.zeros(T, d, dtype=torch.float64, device=DEV)

    def matrix(weights, e, K, gate_up):
        codes, scales, whole = weights
        rows = codes.shape[1]
        value = torch.zeros(rows, K, dtype=torch.float64, device=DEV)
        value[:, 0::2], value[:, 1::2] = (codes[e] & 15).double(), (codes[e] >> 4).double()
        sign = 1.0 - 2.0 * (value >= 8)
        m = value % 8              # sign, two exponent bits, one mantissa bit
        value = sign * torch.where(m < 2, m * 0.5, (2 + m % 2) * 2.0 ** (torch.floor(m / 2) - 2))
        per = scales.view(E, -1)[e]
        if gate_up:                # [I/64, K/64, 32, (gate/up) x 2, 4]
            s = per.view(rows // 128, K // 64, 32, 2, 2, 4).permute(3, 0, 4, 2, 1, 5)
        else:                      # [rows/128, K/64, 32, 4, 4]
            s = per.view(rows // 128, K // 64, 32, 4, 4).permute(0, 3, 2, 1, 4)
        s = s.reshape(rows, K // 16).view(torch.float8_e4m3fn).double()
        return value * s.repeat_interleave(16, 1) * whole[e].double()

    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            a = x[t] @ matrix(st["w13"], e, d, True).t()
            h = torch.nn.functional.silu(a[:, :I]) * a[:, I:]
            o = h @ matrix(st["w2"], e, I, False).t()
            y.index_add_(0, t, o * st["scores"][t, j].double()[:, None])
    return y
