"""Measured cases of a mixture of experts: routing, the experts' feed-forward blocks, and products with 4-bit weights.

Each case is one pass through one operator as a training or serving program
calls it.  ``run`` computes it in plain elementary torch operations in 32 bits
(``own`` false; the order of experts in 64) or through the library's public
functions (``own`` true); ``exact`` computes the same outputs from the
definitions in 64 bits.
"""

import math

import torch

own = False

_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # One step of a served batch, 32 sequences: latency of the call.
        {"name": "route_step", "op": "route", "tokens": 32, "experts": 128, "top": 8, "dtype": "f32",
         "scoring": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_scores": 1, "renorm": True, "scale": 1.0},
        # A prompt, or a training batch: sigmoid scores, a bias for balance, half of the groups of experts.
        {"name": "route_prompt", "op": "route", "tokens": 8192, "experts": 256, "top": 8, "dtype": "f32",
         "scoring": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_scores": 2, "renorm": True, "scale": 2.5},
        # The gradient of a training batch's logits, softmax scores as they are: every logit gets one.
        {"name": "route_grad_train", "op": "route_grad", "tokens": 8192, "experts": 64, "top": 6, "dtype": "bf16",
         "scoring": "softmax", "renorm": False, "scale": 1.0},
        # A small odd batch, renormalised sigmoid scores: few logits get one, all others zero.
        {"name": "route_grad_odd", "op": "route_grad", "tokens": 1001, "experts": 100, "top": 3, "dtype": "f32",
         "scoring": "sigmoid", "renorm": True, "scale": 2.0},
        # One token served: eight experts' weights are read.
        {"name": "experts_token", "op": "experts", "tokens": 1, "experts": 64, "top": 8, "width": 2048, "hidden": 1024,
         "dtype": "bf16", "act": "silu", "save": False},
        # A served batch: nearly every expert has a few tokens.
        {"name": "experts_batch", "op": "experts", "tokens": 48, "experts": 32, "top": 4, "width": 4096, "hidden": 1536,
         "dtype": "f16", "act": "gelu", "save": False},
        # A training batch of 8192 tokens, activations kept for the backward pass.
        {"name": "experts_train", "op": "experts", "tokens": 8192, "experts": 32, "top": 4, "width": 4096, "hidden": 2048,
         "dtype": "bf16", "act": "silu", "save": True},
        # The backward pass of a training batch over many small experts.
        {"name": "experts_grad", "op": "experts_grad", "tokens": 8192, "experts": 64, "top": 6, "width": 2048,
         "hidden": 1408, "dtype": "bf16", "act": "silu"},
        # A small ragged backward pass: no size is a multiple of a tile.
        {"name": "experts_grad_ragged", "op": "experts_grad", "tokens": 517, "experts": 9, "top": 2, "width": 520,
         "hidden": 1048, "dtype": "f16", "act": "gelu"},
        # One token through a large projection with 4-bit weights.
        {"name": "w4_token", "op": "w4", "tokens": 1, "rows": 16384, "width": 8192, "group": 128, "zeros": False,
         "dtype": "bf16"},
        # A small batch, zero points, groups of 64, an odd number of outputs.
        {"name": "w4_batch", "op": "w4", "tokens": 12, "rows": 5001, "width": 4096, "group": 64, "zeros": True,
         "dtype": "f16"},
        # A served step through experts with 4-bit weights: each token with its own four matrices.
        {"name": "w4_experts", "op": "w4", "tokens": 4, "rows": 2048, "width": 2048, "group": 128, "zeros": False,
         "dtype": "bf16", "experts": 32, "top": 4},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "experts", "experts", "experts_grad", "experts_grad", "w4", "w4"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        experts = groups * _log_int(rng, 4, 512 // groups)
        top_groups = rng.randint(1, groups)
        case = {"op": op, "tokens": _log_int(rng, 1, 16384), "experts": experts,
                "top": rng.randint(1, min(8, experts // groups * top_groups)), "dtype": rng.choice(["f32", "bf16", "f16"]),
                "scoring": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 1.0, 2.5])}
        if op == "route_grad" and case["top"] == 1:
            case["renorm"] = False  # one renormalised weight is constant: its gradient is zero and says nothing
        if op == "route":
            case.update(bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, group_scores=rng.choice([1, 2]))
        return case
    if op == "w4":
        group = rng.choice([32, 64, 128])
        while True:
            case = {"op": op, "tokens": _log_int(rng, 1, 32), "rows": _log_int(rng, 64, 16384),
                    "width": group * _log_int(rng, 2, 16384 // group), "group": group, "zeros": rng.random() < 0.5,
                    "dtype": rng.choice(["bf16", "f16"])}
            if rng.random() < 0.4:
                case.update(experts=rng.choice([4, 8, 16, 31]), top=rng.choice([1, 2, 4]))
            if _w4_read(case) * case["rows"] * case["width"] <= 16384 * 8192:
                return case
    while True:
        experts = _log_int(rng, 2, 64)
        case = {"op": op, "tokens": _log_int(rng, 1, 8192), "experts": experts, "top": rng.randint(1, min(8, experts)),
                "width": 8 * _log_int(rng, 16, 512), "hidden": 8 * _log_int(rng, 16, 512),
                "dtype": rng.choice(["bf16", "f16"]), "act": rng.choice(["silu", "gelu", "relu"])}
        size = case["width"] * case["hidden"]
        # no more products than the largest training batch, no more weights than its experts have
        if case["tokens"] * case["top"] * size * (2 if op == "experts_grad" else 1) <= 8192 * 4 * 4096 * 2048 and \
                experts * size <= 32 * 4096 * 2048:
            break
    if op == "experts":
        case["save"] = case["tokens"] > 256 and rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale + shift).to(dtype)

    def chosen(tokens, experts, top):
        """Distinct experts for each token, some experts liked better than others, and weights that sum to one."""
        liking = torch.randn(tokens, experts, device="cuda", generator=gen) + \
            0.5 * torch.randn(experts, device="cuda", generator=gen)
        best = liking.topk(top, dim=1)
        return best.indices.to(torch.int32), torch.softmax(best.values, 1)

    s = {"case": case}
    op, tokens = case["op"], case["tokens"]
    if op in ("route", "route_grad"):
        s["logits"] = normal(tokens, case["experts"], scale=1.5)
        if case.get("bias"):
            s["bias"] = normal(case["experts"], scale=0.1, dtype=torch.float32)
        if op == "route_grad":
            s["experts"] = s["logits"].float().topk(case["top"], dim=1).indices.to(torch.int32)
            s["dweights"] = normal(tokens, case["top"], dtype=torch.float32)
        return s
    if op == "w4":
        rows, width, group = case["rows"], case["width"], case["group"]
        lead = (case["experts"],) if "experts" in case else ()
        s["packed"] = torch.randint(0, 256, (*lead, rows, width // 2), dtype=torch.uint8, device="cuda", generator=gen)
        s["scales"] = (0.01 + 0.02 * torch.rand(*lead, rows, width // group, device="cuda", generator=gen)).to(dt)
        s["zeros"] = torch.randint(4, 12, (*lead, rows, width // group), dtype=torch.uint8, device="cuda",
                                   generator=gen) if case["zeros"] else None
        s["x"] = normal(tokens, width)
        s["experts"] = chosen(tokens, case["experts"], case["top"])[0] if lead else None
        return s
    E, D, F = case["experts"], case["width"], case["hidden"]
    s["x"] = normal(tokens, D)
    s["experts"], s["weights"] = chosen(tokens, E, case["top"])
    s["wg"] = normal(E, F, D, scale=D ** -0.5)
    s["wu"] = normal(E, F, D, scale=D ** -0.5)
    s["wd"] = normal(E, D, F, scale=F ** -0.5)
    if op == "experts_grad":
        s["dy"] = normal(tokens, D)
        # what the forward pass left, a row for each pair of a token and an expert, by expert
        flat = s["experts"].reshape(-1).long()
        order = torch.sort(flat, stable=True).indices
        rows = s["x"][order // case["top"]]
        counts = torch.bincount(flat, minlength=E).tolist()
        s["g"] = torch.cat([r @ w.T for r, w in zip(rows.split(counts), s["wg"])])
        s["u"] = torch.cat([r @ w.T for r, w in zip(rows.split(counts), s["wu"])])
        s["h"] = (_act(s["g"].float(), case["act"]) * s["u"].float()).to(dt)
    return s


# ------------------------------------------------------------------ plain form, 32 bits

def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return torch.where(g > 0, g, torch.zeros_like(g))


def _act_grad(g, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return sig * (1 + g * (1 - sig))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    return (g > 0).to(g.dtype)


def _scores(logits, scoring):
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    case, logits = s["case"], s["logits"]
    groups = case["groups"]
    # The order of the experts is that of exact scores: 64 bits, and without a bias or sums the logits themselves.
    keys = logits.double()
    if case["bias"] or (groups > 1 and case["group_scores"] == 2):
        keys = _scores(keys, case["scoring"])
        if case["bias"]:
            keys = keys + s["bias"].double()
    if groups > 1:
        of_group = keys.reshape(len(keys), groups, -1)
        best = of_group.sort(2, descending=True).values[:, :, :case["group_scores"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter(1, kept, True)
        keys = torch.where(allowed[:, :, None], of_group, torch.full_like(of_group, -math.inf)).reshape(keys.shape)
    chosen = keys.sort(dim=1, descending=True, stable=True).indices[:, :case["top"]]
    w = _scores(logits.float(), case["scoring"]).gather(1, chosen)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return w * case["scale"], chosen.to(torch.int32)


def _plain_route_grad(s):
    case, chosen, dw = s["case"], s["experts"].long(), s["dweights"]
    p = _scores(s["logits"].float(), case["scoring"])
    w = p.gather(1, chosen)
    total = w.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(w[:, :1])
    ds = dw * (case["scale"] / total)
    if case["renorm"]:
        ds = ds - (dw * w).sum(1, keepdim=True) * (case["scale"] / (total * total))
    if case["scoring"] == "sigmoid":
        return torch.zeros_like(p).scatter_add(1, chosen, ds * w * (1 - w)).to(s["logits"].dtype)
    dp = torch.zeros_like(p).scatter_add(1, chosen, ds)
    return (p * (dp - (dp * p).sum(1, keepdim=True))).to(s["logits"].dtype)


def _plain_w4(s):
    x, packed, scales, zeros = s["x"], s["packed"], s["scales"], s["zeros"]
    if s["experts"] is not None:
        packed, scales = packed[s["experts"].long()], scales[s["experts"].long()]
        zeros = zeros[s["experts"].long()] if zeros is not None else None
    q = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).float()
    q = q.reshape(*scales.shape, -1) - (zeros.float()[..., None] if zeros is not None else 8.0)
    w = (q * scales.float()[..., None]).flatten(-2)
    if s["experts"] is None:
        return (x.float() @ w.T).to(x.dtype)
    return (w @ x.float()[:, None, :, None])[..., 0].to(x.dtype)


def _by_expert(s):
    """Pairs of a token and an expert by expert: their order, expert, token, and place among the expert's pairs."""
    flat = s["experts"].reshape(-1).long()
    sorted_, order = torch.sort(flat, stable=True)
    counts = torch.bincount(flat, minlength=s["case"]["experts"])
    place = torch.arange(len(flat), device=flat.device) - (counts.cumsum(0) - counts)[sorted_]
    return order, sorted_, order // s["case"]["top"], place, int(counts.max())


def _plain_experts(s):
    case, x, dt = s["case"], s["x"].float(), s["x"].dtype
    tokens, top, act = case["tokens"], case["top"], case["act"]
    if tokens * top <= case["experts"] and not case["save"]:  # few pairs: the chosen experts' weights alone
        flat = s["experts"].reshape(-1).long()
        rows = x.repeat_interleave(top, 0)[:, :, None]
        h = _act(s["wg"][flat].float() @ rows, act) * (s["wu"][flat].float() @ rows)
        ys = (s["wd"][flat].float() @ h)[:, :, 0]
        return (ys.reshape(tokens, top, -1) * s["weights"][:, :, None]).sum(1).to(dt)
    order, expert, token, place, most = _by_expert(s)
    xs = x.new_zeros(case["experts"], most, x.shape[1])
    xs[expert, place] = x[token]
    g, u = xs @ s["wg"].float().transpose(1, 2), xs @ s["wu"].float().transpose(1, 2)
    h = _act(g, act) * u
    ys = torch.empty(tokens * top, x.shape[1], device=x.device)
    ys[order] = (h @ s["wd"].float().transpose(1, 2))[expert, place]
    y = (ys.reshape(tokens, top, -1) * s["weights"][:, :, None]).sum(1).to(dt)
    return (y, g[expert, place].to(dt), u[expert, place].to(dt), h[expert, place].to(dt)) if case["save"] else y


def _plain_experts_grad(s):
    case, x, dt = s["case"], s["x"].float(), s["x"].dtype
    tokens, top, act = case["tokens"], case["top"], case["act"]
    order, expert, token, place, most = _by_expert(s)

    def padded(rows):
        t = rows.new_zeros(case["experts"], most, rows.shape[1])
        t[expert, place] = rows
        return t

    xs, dys, w = padded(x[token]), padded(s["dy"].float()[token]), padded(s["weights"].reshape(-1, 1)[order])
    g, u, h = padded(s["g"].float()), padded(s["u"].float()), padded(s["h"].float())
    dh = dys @ s["wd"].float()
    dweights = torch.empty(tokens * top, device=x.device)
    dweights[order] = (dh * h).sum(2)[expert, place]
    dh = dh * w
    dg, du = dh * u * _act_grad(g, act), dh * _act(g, act)
    dxs = torch.empty(tokens * top, x.shape[1], device=x.device)
    dxs[order] = (dg @ s["wg"].float() + du @ s["wu"].float())[expert, place]
    dx = dxs.reshape(tokens, top, -1).sum(1)
    return (dx.to(dt), dweights.reshape(tokens, top), (dg.transpose(1, 2) @ xs).to(dt), (du.transpose(1, 2) @ xs).to(dt),
            ((dys * w).transpose(1, 2) @ h).to(dt))


def _plain(s):
    return {"route": _plain_route, "route_grad": _plain_route_grad, "w4": _plain_w4, "experts": _plain_experts,
            "experts_grad": _plain_experts_grad}[s["case"]["op"]](s)


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import software_pipelined_tiled_02_gb300 as tg

    case, op = s["case"], s["case"]["op"]
    if op == "route":
        return tg.route(s["logits"], case["top"], case["scoring"], bias=s.get("bias"), groups=case["groups"],
                        top_groups=case["top_groups"], group_scores=case["group_scores"], renormalize=case["renorm"],
                        scale=case["scale"])
    if op == "route_grad":
        return tg.route_backward(s["dweights"], s["logits"], s["experts"], case["scoring"], renormalize=case["renorm"],
                                 scale=case["scale"])
    if op == "w4":
        return tg.gemm_w4(s["x"], s["packed"], s["scales"], s["zeros"], experts=s["experts"])
    args = (s["x"], s["experts"], s["weights"], s["wg"], s["wu"], s["wd"])
    if op == "experts":
        if not case["save"]:
            return tg.expert_ffn(*args, case["act"])
        y, (g, u, h) = tg.expert_ffn(*args, case["act"], save=True)
        return y, g, u, h
    return tg.expert_ffn_backward(s["dy"], *args, (s["g"], s["u"], s["h"]), case["act"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions, 64 bits

def _exact_route(case, d):
    logits = d["logits"]
    p = torch.softmax(logits, 1) if case["scoring"] == "softmax" else torch.sigmoid(logits)
    keys = p + d["bias"] if case["bias"] else p if case["groups"] > 1 and case["group_scores"] == 2 else logits
    index = torch.arange(keys.shape[1], device=keys.device)

    def largest(values):  # the lowest index of the largest value
        top = values.amax(1, keepdim=True)
        return torch.where(values == top, index[:values.shape[1]], values.shape[1]).amin(1, keepdim=True)

    if case["groups"] > 1:
        size = case["experts"] // case["groups"]
        parts = keys.split(size, 1)
        best = torch.stack([part.topk(min(size, case["group_scores"]), 1).values.sum(1) for part in parts], 1)
        open_ = torch.zeros_like(keys, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            i = largest(best)
            best = best.scatter(1, i, -math.inf)
            open_ |= index // size == i
        keys = keys.masked_fill(~open_, -math.inf)
    chosen = []
    for _ in range(case["top"]):
        chosen.append(largest(keys))
        keys = keys.scatter(1, chosen[-1], -math.inf)
    chosen = torch.cat(chosen, 1)
    w = p.gather(1, chosen)
    return (w / w.sum(1, keepdim=True) if case["renorm"] else w) * case["scale"], chosen.to(torch.int32)


def _exact_route_grad(case, d, chosen):
    z = d["logits"].requires_grad_()
    p = torch.softmax(z, 1) if case["scoring"] == "softmax" else torch.sigmoid(z)
    w = p.gather(1, chosen.long())
    w = (w / w.sum(1, keepdim=True) if case["renorm"] else w) * case["scale"]
    return torch.autograd.grad(w, z, d["dweights"])[0]


def _exact_w4(case, s):
    x, group = s["x"].double(), case["group"]

    def weights(e):
        packed, scales = s["packed"][e], s["scales"][e].double()
        q = torch.empty(packed.shape[0], 2 * packed.shape[1], dtype=torch.float64, device=x.device)
        q[:, 0::2], q[:, 1::2] = packed % 16, packed // 16
        z = s["zeros"][e].double() if s["zeros"] is not None else torch.full_like(scales, 8)
        return (q - z.repeat_interleave(group, 1)) * scales.repeat_interleave(group, 1)

    if s["experts"] is None:
        return x @ weights(slice(None)).T
    chosen = s["experts"].long()
    y = x.new_zeros(*chosen.shape, case["rows"])
    for e in chosen.unique().tolist():
        t, j = (chosen == e).nonzero(as_tuple=True)
        y[t, j] = x[t] @ weights(e).T
    return y


def _normal_cdf(g):
    return 0.5 * torch.special.erfc(-g / math.sqrt(2.0))


def _exact_experts(case, s):
    act, grad = case["act"], case["op"] == "experts_grad"
    x, w = s["x"].double(), s["weights"].double()
    y, dw = torch.zeros_like(x), torch.zeros_like(w)
    kept, dweights = {"g": [], "u": [], "h": []}, {"wg": [], "wu": [], "wd": []}
    row = 0
    for e in range(case["experts"]):
        t, j = (s["experts"] == e).nonzero(as_tuple=True)
        wg, wu, wd = (s[k][e].double() for k in ("wg", "wu", "wd"))
        rows = slice(row, row + len(t))
        row += len(t)
        g, u = (s["g"][rows].double(), s["u"][rows].double()) if grad else (x[t] @ wg.T, x[t] @ wu.T)
        if act == "silu":
            sig = torch.sigmoid(g)
            a, slope = g * sig, sig + g * sig * torch.sigmoid(-g)
        elif act == "gelu":
            a, slope = g * _normal_cdf(g), _normal_cdf(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        else:
            a, slope = g.clamp(min=0), torch.heaviside(g, torch.zeros_like(g))
        if not grad:
            h = a * u
            y.index_add_(0, t, (h @ wd.T) * w[t, j][:, None])
            if case["save"]:
                for k, v in zip("guh", (g, u, h)):
                    kept[k].append(v.float())  # rounded far below the outputs' own type
            continue
        h, dy = s["h"][rows].double(), s["dy"][t].double()
        dh = dy @ wd
        dw[t, j] = (dh * h).sum(1)
        dh = dh * w[t, j][:, None]
        du, dg = dh * a, dh * u * slope
        y.index_add_(0, t, dg @ wg + du @ wu)
        for k, v in (("wg", dg.T @ x[t]), ("wu", du.T @ x[t]), ("wd", (dy * w[t, j][:, None]).T @ h)):
            dweights[k].append(v.float())
    if grad:
        return y, dw, *(torch.stack(v) for v in dweights.values())
    return (y, *(torch.cat(v) for v in kept.values())) if case["save"] else y


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if case["op"] == "route":
        return _exact_route(case, d)
    if case["op"] == "route_grad":
        return _exact_route_grad(case, d, s["experts"])
    if case["op"] == "w4":
        return _exact_w4(case, s)
    return _exact_experts(case, s)


# ------------------------------------------------------------------ the work that cannot be left out

def _w4_read(case):
    """Matrices read: one, or as many as differ among the tokens' choices."""
    return _read(case["tokens"], case["experts"], case["top"]) if "experts" in case else 1.0


def _read(tokens, experts, top):
    """Experts that `tokens` tokens with `top` each are expected to reach."""
    return experts * (1 - (1 - top / experts) ** tokens)


def work(case):
    op, e, t = case["op"], _BYTES[case["dtype"]], case["tokens"]
    if op == "route":
        E, k = case["experts"], case["top"]
        return {"bytes": t * E * e + 8 * t * k + (4 * E if case["bias"] else 0), "flops": 6 * t * E}
    if op == "route_grad":
        E, k = case["experts"], case["top"]
        read = E if case["scoring"] == "softmax" and not case["renorm"] else k
        return {"bytes": t * (E + read) * e + 8 * t * k, "flops": 6 * t * read}
    if op == "w4":
        n, k = case["rows"], case["width"]
        groups, pairs = n * (k // case["group"]), t * case.get("top", 1)
        return {"bytes": _w4_read(case) * (n * k // 2 + groups * (e + (1 if case["zeros"] else 0))) + e * (t * k + pairs * n),
                "flops": 2 * pairs * n * k}
    pairs, d, f = t * case["top"], case["width"], case["hidden"]
    weights = 3 * d * f * e
    read = _read(t, case["experts"], case["top"]) * weights
    if op == "experts":
        return {"bytes": read + e * (2 * t * d + (3 * pairs * f if case["save"] else 0)) + 8 * pairs, "flops": 6 * pairs * d * f}
    return {"bytes": read + case["experts"] * weights + e * (3 * t * d + 3 * pairs * f) + 12 * pairs, "flops": 12 * pairs * d * f}
