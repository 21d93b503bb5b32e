"""Measured cases of the feed-forward operators: layer norm, the gated feed-forward block and dropout.

Each case is one pass through one operator as a training or serving program
calls it.  ``run`` computes it in plain elementary torch operations in 32 bits
(``own`` false) or through the library's public functions (``own`` true);
``exact`` computes the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # One token's activation before a decode step: latency of the call.
        {"name": "norm_token", "op": "norm", "rows": 1, "width": 4096, "dtype": "bf16", "weights": "bf16"},
        # A training batch of 8192 tokens, statistics kept for the backward pass.
        {"name": "norm_train", "op": "norm", "rows": 8192, "width": 4096, "dtype": "bf16", "weights": "f32"},
        # Its backward pass, with the reduction of both weight gradients.
        {"name": "norm_grad", "op": "norm_grad", "rows": 8192, "width": 4096, "dtype": "bf16", "weights": "bf16"},
        # A single-precision model of odd width: rows that start on no vector boundary.
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 4000, "width": 3001, "dtype": "f32", "weights": "f32"},
        # Decoding one token: every weight is read once.
        {"name": "ffn_token", "op": "ffn", "tokens": 1, "width": 4096, "hidden": 8192, "dtype": "bf16",
         "act": "silu", "save": False},
        # Decoding a small batch with a small model: latency of the call.
        {"name": "ffn_batch", "op": "ffn", "tokens": 24, "width": 512, "hidden": 2048, "dtype": "f16",
         "act": "gelu", "save": False},
        # A short ragged training batch: no size is a multiple of a tile.
        {"name": "ffn_ragged", "op": "ffn", "tokens": 513, "width": 3000, "hidden": 5000, "dtype": "f16",
         "act": "gelu", "save": True},
        # A training batch of 8192 tokens, activations kept for the backward pass.
        {"name": "ffn_train", "op": "ffn", "tokens": 8192, "width": 4096, "hidden": 8192, "dtype": "bf16",
         "act": "silu", "save": True},
        # Its backward pass: the gradients of the input and of all three weights.
        {"name": "ffn_grad", "op": "ffn_grad", "tokens": 8192, "width": 4096, "hidden": 8192, "dtype": "bf16",
         "act": "silu"},
        # A small ragged backward pass: an odd token count as the reduction length.
        {"name": "ffn_grad_ragged", "op": "ffn_grad", "tokens": 1001, "width": 520, "hidden": 1400, "dtype": "f16",
         "act": "gelu"},
        # Dropout on a block's output and its residual addition, a training batch.
        {"name": "dropout_train", "op": "dropout", "rows": 8192, "width": 4096, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # The same mask on a gradient, odd sizes, single precision.
        {"name": "dropout_grad_odd", "op": "dropout_grad", "rows": 1001, "width": 4097, "dtype": "f32", "p": 0.25},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width with 16-byte rows at 16 bits: a power of two, or an odd multiple of 8."""
    if rng.random() < 0.5:
        return 1 << rng.randint(int(math.log2(low)), int(math.log2(high)))
    return 8 * (2 * _log_int(rng, low // 16, high // 16 - 1) + 1)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "ffn", "ffn", "ffn_grad", "ffn_grad", "dropout", "dropout_grad"])
    if op in ("norm", "norm_grad", "dropout", "dropout_grad"):
        width = _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            width = 64 * max(1, width // 64)
        case = {"op": op, "rows": _log_int(rng, 1, min(65536, (1 << 25) // width)), "width": width,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
        if op in ("norm", "norm_grad"):
            case["weights"] = rng.choice([case["dtype"], "f32"])
        else:
            case["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
            if op == "dropout":
                case["residual"] = rng.random() < 0.5
        return case
    while True:
        tokens, width, hidden = _log_int(rng, 1, 8192), _width(rng, 128, 8192), _width(rng, 128, 16384)
        if tokens * width * hidden <= 8192 * 4096 * 8192:
            break
    case = {"op": op, "tokens": tokens, "width": width, "hidden": hidden, "dtype": rng.choice(["bf16", "f16"]),
            "act": rng.choice(["silu", "gelu", "relu"])}
    if op == "ffn":
        case["save"] = tokens > 256 and rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale + shift).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, width, wt = case["rows"], case["width"], _DTYPES[case["weights"]]
        # a residual stream: channels of different scales, a common offset
        scale = torch.exp(0.5 * torch.randn(width, device="cuda", generator=gen))
        x32 = torch.randn(rows, width, device="cuda", generator=gen) * scale + 0.25
        s["x"] = x32.to(dt)
        s["w"] = normal(width, scale=0.1, shift=1.0, dtype=wt)
        s["b"] = normal(width, scale=0.1, dtype=wt)
        s["eps"] = 1e-5
        if op == "norm_grad":
            s["dy"] = normal(rows, width)
            xf = s["x"].float()
            mean = xf.mean(1, keepdim=True)
            var = (xf - mean).square().mean(1)
            s["mean"], s["rstd"] = mean.reshape(-1).contiguous(), torch.rsqrt(var + s["eps"])
        return s
    if op in ("dropout", "dropout_grad"):
        s["x"] = normal(case["rows"], case["width"])
        if case.get("residual"):
            s["res"] = normal(case["rows"], case["width"])
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ (seed * 2654435761), (1 << 33) + seed
        return s
    tokens, width, hidden = case["tokens"], case["width"], case["hidden"]
    s["x"] = normal(tokens, width)
    s["wg"] = normal(hidden, width, scale=width ** -0.5)
    s["wu"] = normal(hidden, width, scale=width ** -0.5)
    s["wd"] = normal(width, hidden, scale=hidden ** -0.5)
    if op == "ffn_grad":
        s["dy"] = normal(tokens, width)
        # what the forward pass left: the projections and their gated product
        s["g"] = s["x"] @ s["wg"].T
        s["u"] = s["x"] @ s["wu"].T
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


def _philox_words(n, seed, offset, device):
    """Words 0 .. n-1 of the counter-based generator Philox4x32 with 10 rounds (Salmon et al., 2011):
    counter (block lo, block hi, offset lo, offset hi), key (seed lo, seed hi), four words a block."""
    low = 0xFFFFFFFF
    block = torch.arange((n + 3) // 4, dtype=torch.int64, device=device)
    c0, c1 = block & low, block >> 32
    c2, c3 = torch.full_like(block, offset & low), torch.full_like(block, (offset >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for r in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the products' 64 bits, wrapped into the signed range
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], 1).reshape(-1)[:n]


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dt = s["x"].dtype
    x = s["x"].float()
    if op == "norm":
        mean = x.sum(1, keepdim=True) / case["width"]
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).sum(1, keepdim=True) / case["width"] + s["eps"])
        y = d * rstd * s["w"].float() + s["b"].float()
        return y.to(dt), mean.reshape(-1), rstd.reshape(-1)
    if op == "norm_grad":
        dy, w = s["dy"].float(), s["w"].float()
        rstd = s["rstd"][:, None]
        xh = (x - s["mean"][:, None]) * rstd
        q = dy * w
        dx = rstd * (q - q.sum(1, keepdim=True) / case["width"] - xh * ((q * xh).sum(1, keepdim=True) / case["width"]))
        return dx.to(dt), (dy * xh).sum(0).to(s["w"].dtype), dy.sum(0).to(s["w"].dtype)
    if op in ("dropout", "dropout_grad"):
        words = _philox_words(x.numel(), s["seed"], s["offset"], x.device).reshape(x.shape)
        y = torch.where(words >= int(round(case["p"] * 2.0 ** 32)), x * (1 / (1 - case["p"])), torch.zeros_like(x))
        if "res" in s:
            y = y + s["res"].float()
        return y.to(dt)
    wg, wu, wd = s["wg"].float(), s["wu"].float(), s["wd"].float()
    if op == "ffn":
        g, u = x @ wg.T, x @ wu.T
        h = _act(g, case["act"]) * u
        y = (h @ wd.T).to(dt)
        return (y, g.to(dt), u.to(dt), h.to(dt)) if case["save"] else y
    dy, g, u, h = s["dy"].float(), s["g"].float(), s["u"].float(), s["h"].float()
    dh = dy @ wd
    dg = dh * u * _act_grad(g, case["act"])
    du = dh * _act(g, case["act"])
    dx = dg @ wg + du @ wu
    return dx.to(dt), (dg.T @ x).to(dt), (du.T @ x).to(dt), (dy.T @ h).to(dt)


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import software_pipelined_tiled_02_gb300 as tg

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        return tg.layer_norm(s["x"], s["w"], s["b"], s["eps"], stats=True)
    if op == "norm_grad":
        return tg.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "dropout":
        return tg.dropout(s["x"], case["p"], s["seed"], s["offset"], residual=s.get("res"))
    if op == "dropout_grad":
        return tg.dropout_backward(s["x"], case["p"], s["seed"], s["offset"])
    if op == "ffn":
        if not case["save"]:
            return tg.gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], case["act"])
        y, (g, u, h) = tg.gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], case["act"], save=True)
        return y, g, u, h
    return tg.gated_ffn_backward(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], (s["g"], s["u"], s["h"]), case["act"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions, 64 bits

def _normal_cdf(g):
    return 0.5 * torch.special.erfc(-g / math.sqrt(2.0))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "norm":
        mean = d["x"].mean(1)
        rstd = (d["x"].var(1, unbiased=False) + s["eps"]).rsqrt()
        return torch.addcmul(d["b"], (d["x"] - mean[:, None]) * rstd[:, None], d["w"]), mean, rstd
    if op == "norm_grad":
        xh = (d["x"] - d["mean"][:, None]) * d["rstd"][:, None]
        q = d["dy"] * d["w"]
        along = (q * xh).mean(1, keepdim=True)
        return (q - q.mean(1, keepdim=True) - along * xh) * d["rstd"][:, None], torch.einsum("ij,ij->j", d["dy"], xh), \
            d["dy"].sum(0)
    if op in ("dropout", "dropout_grad"):
        n = d["x"].numel()
        if n > 1 << 26:
            return None  # the generator below works through the elements on the host
        import numpy as np

        m32 = np.uint64(0xFFFFFFFF)
        b = np.arange((n + 3) // 4, dtype=np.uint64)
        off, key = s["offset"], s["seed"]
        ctr = [b & m32, b >> np.uint64(32), np.full_like(b, off & 0xFFFFFFFF), np.full_like(b, (off >> 32) & 0xFFFFFFFF)]
        for r in range(10):
            k = [np.uint64(((key & 0xFFFFFFFF) + r * 0x9E3779B9) & 0xFFFFFFFF),
                 np.uint64((((key >> 32) & 0xFFFFFFFF) + r * 0xBB67AE85) & 0xFFFFFFFF)]
            a, c = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
            ctr = [(c >> np.uint64(32)) ^ ctr[1] ^ k[0], c & m32, (a >> np.uint64(32)) ^ ctr[3] ^ k[1], a & m32]
        u = np.stack(ctr, 1).reshape(-1)[:n]
        kept = torch.from_numpy(u >= np.uint64(int(round(case["p"] * 2.0 ** 32)))).to("cuda").reshape(d["x"].shape)
        y = d["x"] * kept / (1 - case["p"])
        return y + d["res"] if "res" in d else y
    act = case["act"]
    if op == "ffn":
        g, u = d["x"] @ d["wg"].T, d["x"] @ d["wu"].T
        a = g * torch.sigmoid(g) if act == "silu" else g * _normal_cdf(g) if act == "gelu" else g.clamp(min=0)
        h = a * u
        y = h @ d["wd"].T
        return (y, g, u, h) if case["save"] else y
    g, u = d["g"], d["u"]
    if act == "silu":
        sig = torch.sigmoid(g)
        a, slope = g * sig, sig + g * sig * torch.sigmoid(-g)
    elif act == "gelu":
        a, slope = g * _normal_cdf(g), _normal_cdf(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        a, slope = g.clamp(min=0), torch.heaviside(g, torch.zeros_like(g))
    dh = d["dy"] @ d["wd"]
    du, dg = dh * a, dh * u * slope
    return dg @ d["wg"] + du @ d["wu"], dg.T @ d["x"], du.T @ d["x"], d["dy"].T @ d["h"]


# ------------------------------------------------------------------ the work that cannot be left out

def work(case):
    op, e = case["op"], _BYTES[case["dtype"]]
    if op in ("norm", "norm_grad"):
        n, w = case["rows"] * case["width"], _BYTES[case["weights"]] * case["width"]
        if op == "norm":
            return {"bytes": 2 * n * e + 2 * w + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * w + 8 * case["rows"], "flops": 14 * n}
    if op in ("dropout", "dropout_grad"):
        n = case["rows"] * case["width"]
        return {"bytes": (3 if case.get("residual") else 2) * n * e, "flops": 3 * n}
    t, d, f = case["tokens"], case["width"], case["hidden"]
    if op == "ffn":
        return {"bytes": e * (2 * t * d + 3 * d * f + (3 * t * f if case["save"] else 0)), "flops": 6 * t * d * f}
    return {"bytes": e * (3 * t * d + 3 * t * f + 6 * d * f), "flops": 12 * t * d * f}
