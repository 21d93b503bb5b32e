"""Plain 64-bit forms of the mixture-of-experts operators and the error bounds
their tests use.  Nothing here uses the product's code."""

import math

import torch

from tests import operator_reference as ref

U = ref.U


def scores(logits, scoring):
    """Scores of every expert; zeros for a row whose logits are all -inf."""
    l = logits.double()
    if scoring == "sigmoid":
        return torch.sigmoid(l)
    return torch.where(torch.isneginf(l).all(1, keepdim=True), torch.zeros_like(l), torch.softmax(l, 1))


def choose(keys, count):
    """Indices of the `count` largest keys of one row, ties to the lowest index, NaN above all."""
    order = sorted(range(len(keys)), key=lambda i: (0 if keys[i] != keys[i] else 1, -keys[i] if keys[i] == keys[i] else 0, i))
    return order[:count]


def route(logits, top, scoring="softmax", bias=None, groups=1, top_groups=None, group_scores=1, renormalize=True, scale=1.0):
    """(weights in 64 bits, experts) by the definition, row by row on the host."""
    logits = logits.cpu()
    s = scores(logits, scoring)
    top_groups = top_groups or groups
    chosen = []
    for t in range(len(logits)):
        keys = s[t] + bias.cpu().double() if bias is not None else logits[t].double()
        open_ = range(len(keys))
        if top_groups < groups:
            size = len(keys) // groups
            from_ = keys if bias is not None else s[t] if group_scores == 2 else keys
            totals = [sum(sorted(from_[g * size:(g + 1) * size].tolist(), reverse=True)[:group_scores]) for g in range(groups)]
            best = choose(totals, top_groups)
            open_ = [e for e in open_ if e // size in best]
        keys = keys.tolist()
        picked = choose([keys[e] for e in open_], top)
        chosen.append([open_[i] for i in picked])
    chosen = torch.tensor(chosen, dtype=torch.int64).reshape(len(logits), top)
    return weights_of(logits, chosen, scoring, renormalize, scale), chosen


def weights_of(logits, chosen, scoring, renormalize, scale):
    """Weights of given choices; -1 marks an entry that takes no part."""
    s = scores(logits, scoring).gather(1, chosen.clamp(min=0)) * (chosen >= 0)
    if renormalize:
        l = logits.double().gather(1, chosen.clamp(min=0))
        l = torch.where(chosen >= 0, l, torch.full_like(l, -math.inf))
        log_s = l if scoring == "softmax" else torch.nn.functional.logsigmoid(l)  # no underflow before the quotient
        s = torch.where(torch.isneginf(log_s).all(1, keepdim=True), torch.zeros_like(l), torch.softmax(log_s, 1))
    return s * scale


def weight_bound(logits, w):
    """Relative errors: expf 4 U, its argument's rounding U (largest - l) for each term and for the sum, whose mean
    of that is below the largest; 40 U for sums over lanes and registers, quotients and the scale."""
    spread = torch.nan_to_num(logits.double(), neginf=0.0).abs().amax(1, keepdim=True) * 2
    return w.abs() * U * (60 + 4 * spread) + 2.0 ** -120


def route_backward(dweights, logits, chosen, scoring="softmax", renormalize=True, scale=1.0):
    """(dlogits, sum of the magnitudes that meet in each) from the formulas."""
    dw = dweights.double()
    ok = chosen >= 0
    at = chosen.clamp(min=0)
    dw = dw * ok
    s = scores(logits, scoring)
    out, mag = torch.zeros_like(s), torch.zeros_like(s)
    if scoring == "softmax" and not renormalize:
        p = s.gather(1, at)
        q, qm = (p * dw).sum(1, keepdim=True), (p * dw).abs().sum(1, keepdim=True)
        out -= scale * s * q
        mag += scale * s * qm
        out.scatter_add_(1, at, scale * p * dw)
        mag.scatter_add_(1, at, scale * (p * dw).abs())
        return out, mag
    slope = torch.sigmoid(-logits.double()).gather(1, at) if scoring == "sigmoid" else torch.ones_like(dw)
    if renormalize:
        p = weights_of(logits, chosen, scoring, True, 1.0)
        q, qm = (p * dw).sum(1, keepdim=True), (p * dw).abs().sum(1, keepdim=True)
        part, m = scale * p * (dw - q) * slope, scale * p * (dw.abs() + qm) * slope
    else:
        part = scale * s.gather(1, at) * dw * slope
        m = part.abs()
    out.scatter_add_(1, at, part * ok)
    mag.scatter_add_(1, at, m * ok)
    return out, mag


def unpack_w4(packed, scales, zeros):
    """Weights in 64 bits."""
    q = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).double()
    q = q.reshape(*scales.shape, -1)
    z = zeros.double()[..., None] if zeros is not None else 8.0
    return ((q - z) * scales.double()[..., None]).flatten(-2)
