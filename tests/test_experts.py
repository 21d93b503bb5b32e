"""The experts' feed-forward blocks on the GPU against their 64-bit definition.

Bounds: each pair's g, u and h as in tests/test_ffn.py; its share of y is off by
what h's bound and the second product's sum allow, times its weight, and a
token's sum over its pairs by U for each.  The gradients likewise: dg and du
carry the weight's rounding on top, dw_down's operand w h one rounding to 16
bits, and a pair's dweight, which is not rounded to 16 bits, the fp32 sum over
the hidden units: mm(width) of dh's magnitudes and (hidden / 32 + 64) U.
"""

import pytest
import torch

from tests import operator_reference as ref
from tests.test_ffn import DT, U, mm, rounding, within

ACTS = ["silu", "gelu", "relu"]


def make(seed, tokens, experts, top, width, hidden, dtype, invalid=False, only=None):
    """`only`: the experts that are chosen at all."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    liking = torch.randn(tokens, experts, generator=gen, device="cuda") + torch.randn(experts, generator=gen, device="cuda")
    if only is not None:
        keep = torch.zeros(experts, device="cuda")
        keep[only] = 100.0
        liking = liking + keep
    chosen = liking.topk(top, 1).indices.int()
    if invalid:
        chosen[torch.rand(tokens, top, generator=gen, device="cuda") < 0.2] = -1
        chosen[torch.rand(tokens, top, generator=gen, device="cuda") < 0.1] = experts
    return {"x": normal(tokens, width), "e": chosen, "w": torch.rand(tokens, top, generator=gen, device="cuda") - 0.2,
            "wg": normal(experts, hidden, width, scale=width ** -0.5), "wu": normal(experts, hidden, width, scale=width ** -0.5),
            "wd": normal(experts, width, hidden, scale=hidden ** -0.5), "dy": normal(tokens, width)}


def args(d):
    return d["x"], d["e"], d["w"], d["wg"], d["wu"], d["wd"]


def pairs_of(d):
    """For each expert its pairs' tokens and places, in order."""
    for e in range(len(d["wg"])):
        yield (e, *(d["e"] == e).nonzero(as_tuple=True))


def forward_reference(d, act):
    dt = d["x"].dtype
    x, w = d["x"].double(), d["w"].double()
    y, mag, yb = (torch.zeros_like(x) for _ in range(3))
    saved = {k: [] for k in "guh"}
    for e, t, j in pairs_of(d):
        xe, wg, wu, wd = x[t], d["wg"][e].double(), d["wu"][e].double(), d["wd"][e].double()
        g, u = xe @ wg.T, xe @ wu.T
        gb, ub = mm(x.shape[1]) * (xe.abs() @ wg.abs().T), mm(x.shape[1]) * (xe.abs() @ wu.abs().T)
        a, slope = ref.activation(g, act)
        h = a * u
        ab = slope.abs().clamp(min=1.2) * gb + 64 * U * a.abs() + 8 * U * g.abs()
        hb = u.abs() * ab + (a.abs() + ab) * ub + rounding(h, dt)
        ys = h @ wd.T
        ysb = hb @ wd.abs().T + mm(wd.shape[1]) * ((h.abs() + hb) @ wd.abs().T)
        we = w[t, j][:, None]
        y.index_add_(0, t, we * ys)
        mag.index_add_(0, t, we.abs() * (ys.abs() + ysb))
        yb.index_add_(0, t, we.abs() * ysb)
        for k, v, b in (("g", g, gb + rounding(g, dt)), ("u", u, ub + rounding(u, dt)), ("h", h, hb)):
            saved[k].append((v, b))
    yb = yb + (d["e"].shape[1] + 1) * U * mag
    out = {k: tuple(torch.cat(v) for v in zip(*saved[k])) for k in "guh"}
    out["y"] = (y, yb + rounding(y.abs() + yb, dt))
    return out


def backward_reference(d, saved, act):
    dt = d["x"].dtype
    x, w, dyt = d["x"].double(), d["w"].double(), d["dy"].double()
    F, D = d["wg"].shape[1:]
    dx, dxb, dxm = (torch.zeros_like(x) for _ in range(3))
    dw, dwb = torch.zeros_like(w), torch.zeros_like(w)
    grads = {k: [] for k in ("dw_gate", "dw_up", "dw_down")}
    row = 0
    for e, t, j in pairs_of(d):
        rows = slice(row, row + len(t))
        row += len(t)
        xe, dy, we = x[t], dyt[t], w[t, j][:, None]
        wg, wu, wd = d["wg"][e].double(), d["wu"][e].double(), d["wd"][e].double()
        g, u, h = (s[rows].double() for s in saved)
        a, slope = ref.activation(g, act)
        dh = dy @ wd
        dhb = mm(D) * (dy.abs() @ wd.abs())
        dw[t, j] = (dh * h).sum(1)
        dwb[t, j] = (dhb * h.abs()).sum(1) + (F / 32 + 64) * U * ((dh.abs() + dhb) * h.abs()).sum(1) + 2.0 ** -140
        dhw, dhwb = dh * we, (dhb + U * dh.abs()) * we.abs()
        dg, du = dhw * u * slope, dhw * a
        ab, sb = 64 * U * a.abs() + 8 * U * g.abs(), 64 * U * (1 + g.abs())
        dgb = u.abs() * (slope.abs() * dhwb + (dhw.abs() + dhwb) * sb) + 2 * U * dg.abs() + rounding(dg, dt)
        dub = a.abs() * dhwb + (dhw.abs() + dhwb) * ab + rounding(du, dt)
        hw = h * we
        hwb = rounding(hw, dt) + U * hw.abs()
        dx.index_add_(0, t, dg @ wg + du @ wu)
        m = (dg.abs() + dgb) @ wg.abs() + (du.abs() + dub) @ wu.abs()
        dxb.index_add_(0, t, dgb @ wg.abs() + dub @ wu.abs() + mm(2 * F + 128) * m)
        dxm.index_add_(0, t, m)
        for k, left, lb, right, rb in (("dw_gate", dg, dgb, xe, xe * 0), ("dw_up", du, dub, xe, xe * 0), ("dw_down", dy, dy * 0, hw, hwb)):
            b = lb.abs().T @ (right.abs() + rb) + left.abs().T @ rb.abs() + \
                mm(len(t)) * ((left.abs() + lb).T @ (right.abs() + rb))
            grads[k].append((left.T @ right, b))
    dxb = dxb + (d["e"].shape[1] + 1) * U * dxm
    out = {"dx": (dx, dxb + rounding(dx.abs() + dxb, dt)), "dweights": (dw, dwb)}
    for k, v in grads.items():
        value, b = (torch.stack(s) for s in zip(*v))
        out[k] = (value, b + rounding(value.abs() + b, dt))
    return out


NAMES = ("dx", "dweights", "dw_gate", "dw_up", "dw_down")


def check_forward(tg, d, act, **kw):
    want = forward_reference(d, act)
    y, saved = tg.expert_ffn(*args(d), act, save=True, **kw)
    within(y, *want["y"], "y")
    used = len(want["g"][0])
    for name, t in zip("guh", saved):
        assert t.shape[0] == d["e"].numel()
        within(t[:used], *want[name], name)
    within(tg.expert_ffn(*args(d), act, **kw), *want["y"], "y without save")
    return y, saved


def check_backward(tg, d, saved, act):
    got = tg.expert_ffn_backward(d["dy"], *args(d), saved, act)
    want = backward_reference(d, saved, act)
    for name, t in zip(NAMES, got):
        within(t, *want[name], name)
    return got


# tokens, experts, top, width, hidden
SHAPES = [(1, 1, 1, 8, 8), (1, 4, 2, 64, 72), (2, 64, 8, 128, 64), (5, 3, 3, 72, 200), (8, 8, 2, 264, 520), (9, 40, 8, 128, 256),
          (33, 7, 2, 136, 104), (40, 1, 1, 256, 1000), (64, 32, 4, 512, 136), (100, 5, 4, 520, 264), (257, 2, 1, 96, 1032),
          (300, 16, 6, 328, 648), (700, 3, 2, 264, 520), (1100, 128, 2, 72, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(cuda_lib, shape, act, dtype):
    d = make(sum(shape), *shape, dtype)
    _, saved = check_forward(cuda_lib, d, act)
    check_backward(cuda_lib, d, saved, act)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(3, 5, 2, 64, 72), (50, 6, 3, 128, 264), (900, 12, 4, 136, 328)])
def test_indices_out_of_range_take_no_part(cuda_lib, shape):
    d = make(3, *shape, "bf16", invalid=True)
    d["e"][1] = -1
    y, saved = check_forward(cuda_lib, d, "silu")
    dx, dw, *_ = check_backward(cuda_lib, d, saved, "silu")
    assert not y[1].any() and not dx[1].any() and not dw[1].any()
    d["e"][:] = shape[1] + 7  # none at all
    y, saved = cuda_lib.expert_ffn(*args(d), save=True)
    got = cuda_lib.expert_ffn_backward(d["dy"], *args(d), saved)
    assert not y.any() and not any(t.any() for t in got)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [4, 70, 600])
def test_the_same_expert_twice(cuda_lib, tokens):
    d = make(5, tokens, 9, 4, 136, 264, "bf16")
    d["e"][:, 2] = d["e"][:, 0]
    d["e"][1] = d["e"][1, 0]
    _, saved = check_forward(cuda_lib, d, "gelu")
    check_backward(cuda_lib, d, saved, "gelu")


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,only", [(600, [3]), (1500, [0, 15]), (31, [7]), (2048, [5, 6])])
def test_uneven_experts(cuda_lib, tokens, only):
    """Experts without any token beside one or two that have all, and more pairs than one CTA places."""
    d = make(7, tokens, 16, len(only), 200, 296, "bf16", only=only)
    _, saved = check_forward(cuda_lib, d, "silu")
    got = check_backward(cuda_lib, d, saved, "silu")
    idle = [e for e in range(16) if e not in only]
    assert all(not g[idle].any() and bool(g[only].any()) for g in got[2:])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(4100, 24, 4, 520, 264), (2000, 8, 2, 1032, 2056), (48, 32, 4, 4096, 1536), (1, 64, 8, 2048, 1024),
                                   (5000, 1024, 3, 64, 72), (20, 300, 32, 264, 136), (3, 2, 2, 8192, 264)])
def test_larger_shapes(cuda_lib, shape):
    d = make(9, *shape, "bf16")
    _, saved = check_forward(cuda_lib, d, "silu")
    check_backward(cuda_lib, d, saved, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("only", [None, 40, 11])
@pytest.mark.parametrize("shape", [(30, 64, 8, 136, 72), (12, 260, 32, 72, 136), (48, 200, 8, 264, 200), (20, 9, 1, 64, 520),
                                   (47, 64, 4, 1032, 264)])
def test_a_few_pairs_of_many_experts(cuda_lib, shape, only):
    """Experts without pairs, with several, and with more than one pass of 8 takes."""
    tokens, experts, top = shape[:3]
    d = make(17, *shape, "bf16", invalid=only is None, only=None if only is None else list(range(min(experts, max(only, top)))))
    within(cuda_lib.expert_ffn(*args(d)), *forward_reference(d, "silu")["y"], "y")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 6, 4, 72, 136), (1, 3, 5, 264, 72), (8, 64, 8, 136, 264), (10, 4, 4, 72, 1032)])
def test_tokens_that_choose_alike(cuda_lib, shape):
    """One list of experts for all tokens; the last choice repeats the first, the one before names none."""
    tokens, experts, top, width, hidden = shape
    d = make(19, tokens, experts, min(top, experts), width, hidden, "bf16")
    d["e"] = d["e"][:1, torch.arange(top, device="cuda") % experts].repeat(tokens, 1)
    d["w"] = torch.rand(tokens, top, generator=torch.Generator(device="cuda").manual_seed(20), device="cuda") - 0.2
    d["e"][:, -1] = d["e"][:, 0]
    d["e"][:, -2] = -1
    within(cuda_lib.expert_ffn(*args(d)), *forward_reference(d, "silu")["y"], "y")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(33500, 16, 8, 8, 8), (70000, 260, 4, 16, 8)])
def test_many_chunks_of_pairs(cuda_lib, shape):
    """More chunks than a CTA scans at once, and some indices that name no expert."""
    d = make(13, *shape, "f16", invalid=True)
    _, saved = check_forward(cuda_lib, d, "relu")
    check_backward(cuda_lib, d, saved, "relu")


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [2, 30, 400])
def test_infinities_stay_with_their_tokens(cuda_lib, tokens):
    """A token of infinities and NaN spoils its own result alone, and in training the experts that it chose."""
    d = make(11, tokens, 12, 2, 136, 264, "bf16")
    clean, saved = cuda_lib.expert_ffn(*args(d), save=True)
    want = cuda_lib.expert_ffn_backward(d["dy"], *args(d), saved)
    d["x"][1] = float("nan")
    d["x"][1, ::2] = float("inf")
    y, saved = cuda_lib.expert_ffn(*args(d), save=True)
    got = cuda_lib.expert_ffn_backward(d["dy"], *args(d), saved)
    others = torch.arange(tokens) != 1
    assert torch.equal(y[others], clean[others]) and not y[1].isfinite().any()
    assert torch.equal(got[0][others], want[0][others]) and torch.equal(got[1][others], want[1][others])
    rest = [e for e in range(12) if e not in d["e"][1].tolist()]
    assert all(torch.equal(g[rest], w[rest]) for g, w in zip(got[2:], want[2:]))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [2, 40, 500])
def test_weights_of_other_experts_do_not_matter(cuda_lib, tokens):
    """Experts that nothing chose hold NaN."""
    d = make(13, tokens, 10, 2, 72, 136, "f16", only=[2, 5, 8])
    want_y, saved = cuda_lib.expert_ffn(*args(d), save=True)
    want = cuda_lib.expert_ffn_backward(d["dy"], *args(d), saved)
    idle = [e for e in range(10) if e not in d["e"].unique().tolist()]
    for k in ("wg", "wu", "wd"):
        d[k][idle] = float("nan")
    y, saved = cuda_lib.expert_ffn(*args(d), save=True)
    assert torch.equal(y, want_y)
    assert all(torch.equal(a, b) for a, b in zip(cuda_lib.expert_ffn_backward(d["dy"], *args(d), saved), want))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 5, 2, 64, 72), (40, 5, 2, 72, 136), (300, 6, 3, 136, 264)])
def test_strides_and_streams(cuda_lib, shape):
    tg, d = cuda_lib, make(15, *shape, "bf16")
    want_y, saved = tg.expert_ffn(*args(d), save=True)
    want = tg.expert_ffn_backward(d["dy"], *args(d), saved)
    tokens, experts, top, width, hidden = shape
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, dy = nan(tokens, width + 16)[:, 8:8 + width], nan(tokens, width + 8)[:, :width]
    both = nan(experts, 2 * hidden, width)  # gate and up projection in one tensor
    down = nan(experts, width + 3, hidden + 8)[:, :width, :hidden]
    x.copy_(d["x"])
    dy.copy_(d["dy"])
    both[:, :hidden], both[:, hidden:] = d["wg"], d["wu"]
    down.copy_(d["wd"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = (x, d["e"], d["w"], both[:, :hidden], both[:, hidden:], down)
    y, s = tg.expert_ffn(*a, save=True, stream=side)
    got = tg.expert_ffn_backward(dy, *a, s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want_y) and all(torch.equal(p, q) for p, q in zip((*s, *got), (*saved, *want)))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 8, 2, 64, 72), (40, 9, 2, 136, 264), (1200, 20, 4, 264, 136)])
def test_repeats_and_replays_are_equal(cuda_lib, shape):
    """The same bits each time, and a captured step follows its inputs."""
    tg, d = cuda_lib, make(17, *shape, "bf16")

    def step():
        y, saved = tg.expert_ffn(*args(d), save=True)
        return (y, tg.expert_ffn(*args(d)), *saved, *tg.expert_ffn_backward(d["dy"], *args(d), saved))

    want = step()
    assert all(torch.equal(a, b) for _ in range(3) for a, b in zip(step(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    other = make(18, *shape, "bf16")
    for k in ("x", "e", "w", "dy"):
        d[k].copy_(other[k])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.gpu
def test_no_tokens(cuda_lib):
    d = make(19, 4, 3, 2, 64, 72, "bf16")
    for k in ("x", "e", "w", "dy"):
        d[k] = d[k][:0]
    y, saved = cuda_lib.expert_ffn(*args(d), save=True)
    assert y.shape == (0, 64) and all(t.shape == (0, 72) for t in saved)
    got = cuda_lib.expert_ffn_backward(d["dy"], *args(d), saved)
    assert got[0].shape == (0, 64) and got[1].shape == (0, 2) and not any(t.any() for t in got[2:])


@pytest.mark.gpu
def test_gradients_against_differences(cuda_lib):
    """The formulas of the reference against differences of the 64-bit forward pass, and the kernels against the formulas."""
    d = make(21, 6, 4, 2, 16, 24, "f16")
    _, saved = cuda_lib.expert_ffn(*args(d), "silu", save=True)

    def loss(v):
        y = torch.zeros_like(v["x"])
        for e, t, j in pairs_of(d):
            g, u = v["x"][t] @ v["wg"][e].T, v["x"][t] @ v["wu"][e].T
            y.index_add_(0, t, v["w"][t, j][:, None] * ((torch.nn.functional.silu(g) * u) @ v["wd"][e].T))
        return float((y * d["dy"].double()).sum())

    v = {k: d[k].double() for k in ("x", "w", "wg", "wu", "wd")}
    exact = tuple(torch.cat(s) for s in zip(*((v["x"][t] @ v["wg"][e].T, v["x"][t] @ v["wu"][e].T) for e, t, _ in pairs_of(d))))
    exact = (*exact, torch.nn.functional.silu(exact[0]) * exact[1])
    want = backward_reference(d, exact, "silu")
    gen = torch.Generator().manual_seed(1)
    for key, name in (("x", "dx"), ("w", "dweights"), ("wg", "dw_gate"), ("wu", "dw_up"), ("wd", "dw_down")):
        for _ in range(5):
            at = int(torch.randint(0, v[key].numel(), (1,), generator=gen))
            flat, keep = v[key].view(-1), float(v[key].view(-1)[at])
            flat[at] = keep + 1e-5
            up = loss(v)
            flat[at] = keep - 1e-5
            down = loss(v)
            flat[at] = keep
            assert abs((up - down) / 2e-5 - float(want[name][0].reshape(-1)[at])) < 1e-6
    check_backward(cuda_lib, d, saved, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [32, 300])
def test_saved_rows_behind_the_last_are_left_alone(cuda_lib, rows):
    """Through the C entry points, with bands around every output."""
    tg, d = cuda_lib, make(23, rows, 5, 2, 72, 136, "bf16", invalid=True)
    L, plan, s = tg.load(), tg.GatedFFN(72, 136), torch.cuda.current_stream().cuda_stream
    used = int(((d["e"] >= 0) & (d["e"] < 5)).sum())
    want_y, want = tg.expert_ffn(*args(d), save=True)
    band = 64

    def banded(n, width, dtype=torch.bfloat16):
        return torch.full(((n + 2 * band) * width,), 7.0, dtype=dtype, device="cuda")

    def inner(t, width):
        return t[band * width:-band * width].view(-1, width)

    y, g, u, h = banded(rows, 72), *(banded(2 * rows, 136) for _ in range(3))
    need = L.tgemm_experts_workspace(plan.handle, rows, 5, 2, 1)
    work = torch.zeros(need + 512, dtype=torch.uint8, device="cuda")
    weights = [v for k in ("wg", "wu", "wd") for v in (d[k].data_ptr(), d[k].stride(1), d[k].stride(0))]
    p = lambda t, w: inner(t, w).data_ptr()  # noqa: E731
    assert L.tgemm_experts_forward(plan.handle, rows, 5, 2, d["x"].data_ptr(), 72, d["e"].data_ptr(), d["w"].data_ptr(), *weights,
                                   p(y, 72), 72, p(g, 136), p(u, 136), p(h, 136), work.data_ptr(), need, s) == tg.OK
    torch.cuda.synchronize()
    assert torch.equal(inner(y, 72), want_y) and not work[need:].any()
    for t, v in zip((g, u, h), want):
        assert torch.equal(inner(t, 136)[:used], v[:used]) and bool((inner(t, 136)[used:] == 7).all())
    for t, width in ((y, 72), (g, 136), (u, 136), (h, 136)):
        assert bool((t[:band * width] == 7).all()) and bool((t[-band * width:] == 7).all())
    outs = [banded(rows, 72), banded(rows, 2, torch.float32), banded(5 * 136, 72), banded(5 * 136, 72), banded(5 * 72, 136)]
    widths = [72, 2, 72, 72, 136]
    need = L.tgemm_experts_workspace(plan.handle, rows, 5, 2, 2)
    work = torch.zeros(need + 512, dtype=torch.uint8, device="cuda")
    dx, dw, *dws = (p(t, w) for t, w in zip(outs, widths))
    call = lambda *o: L.tgemm_experts_backward(plan.handle, rows, 5, 2, d["dy"].data_ptr(), 72, d["x"].data_ptr(), 72,  # noqa: E731
                                               d["e"].data_ptr(), d["w"].data_ptr(), *weights, *(t.data_ptr() for t in want), o[0], 72,
                                               o[1], *o[2:], work.data_ptr(), need, s)
    assert call(dx, dw, *dws) == tg.OK
    got = tg.expert_ffn_backward(d["dy"], *args(d), want)
    torch.cuda.synchronize()
    assert not work[need:].any()
    for t, w, v in zip(outs, widths, got):
        assert torch.equal(inner(t, w).reshape(-1), v.reshape(-1))
        assert bool((t[:band * w] == 7).all()) and bool((t[-band * w:] == 7).all())
    # any gradient may be left out
    for i in range(5):
        for t in outs:
            t.fill_(7.0)
        o = [dx, dw, *dws]
        o[i] = None
        assert call(*o) == tg.OK
        torch.cuda.synchronize()
        for k, (t, w, v) in enumerate(zip(outs, widths, got)):
            assert bool((t == 7).all()) if k == i else torch.equal(inner(t, w).reshape(-1), v.reshape(-1))
    assert plan.status()[0] == tg.OK
    plan.close()


def test_refusals_without_a_gpu():
    import software_pipelined_tiled_02_gb300 as tg

    x, w = torch.zeros(2, 8).half(), torch.zeros(1, 8, 8).half()
    with pytest.raises((ValueError, tg.TgemmError)):
        tg.expert_ffn(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), w, w, w)
    with pytest.raises(TypeError):
        tg.expert_ffn([1], None, None, w, w, w)
    with pytest.raises(ValueError):
        tg.expert_ffn(x, None, None, w[0], w[0], w[0])
    L = tg.load()
    assert L.tgemm_experts_workspace(None, 1, 1, 1, 0) == -tg.ERR_INVALID_ARG


@pytest.mark.gpu
def test_refusals(cuda_lib):
    tg, d = cuda_lib, make(25, 6, 4, 2, 64, 72, "bf16")
    _, saved = tg.expert_ffn(*args(d), save=True)

    def bad(kind, **change):
        v = {**d, **change}
        with pytest.raises(kind):
            tg.expert_ffn(*args(v), change.get("act", "silu"))
        with pytest.raises(kind):
            tg.expert_ffn_backward(v["dy"], *args(v), saved, change.get("act", "silu"))

    bad(TypeError, e=d["e"].long())
    bad(TypeError, w=d["w"].half())
    bad(TypeError, wu=d["wu"].half())
    bad(TypeError, wg=None)
    bad(ValueError, e=d["e"][:5])
    bad(ValueError, w=d["w"][:, :1])
    bad(ValueError, e=d["e"][:, :0], w=d["w"][:, :0])
    bad(ValueError, e=d["e"].t().contiguous().t())
    bad(ValueError, e=d["e"].cpu())
    bad(ValueError, wg=d["wg"][:3])
    bad(ValueError, wd=d["wd"].transpose(1, 2))
    bad(ValueError, wu=d["wu"][0])
    bad(ValueError, wu=d["wu"][:1].expand(4, 72, 64))
    bad(ValueError, x=d["x"].cpu())
    bad(ValueError, act="tanh")
    for s in (saved[:2], list(saved), (saved[0], saved[1], None)):
        with pytest.raises(TypeError):
            tg.expert_ffn_backward(d["dy"], *args(d), s)
    for s in ((saved[0][:5], *saved[1:]), (saved[0].t().contiguous().t(), *saved[1:])):
        with pytest.raises(ValueError):
            tg.expert_ffn_backward(d["dy"], *args(d), s)
    with pytest.raises(tg.TgemmError):  # rows off the 16-byte boundary
        tg.expert_ffn(torch.zeros(6 * 64 + 1, device="cuda").bfloat16()[1:].view(6, 64), *args(d)[1:])
    L, plan = tg.load(), tg.GatedFFN(64, 72)
    ws = L.tgemm_experts_workspace
    assert ws(plan.handle, 10, 4, 2, 0) > 0
    for a in ((-1, 4, 2, 0), (10, 0, 2, 0), (10, 1025, 2, 0), (10, 4, 0, 0), (10, 4, 33, 0), (10, 4, 2, 3), (1 << 30, 4, 2, 0)):
        assert ws(plan.handle, *a) == -tg.ERR_INVALID_ARG, a
    weights = [v for k in ("wg", "wu", "wd") for v in (d[k].data_ptr(), d[k].stride(1), d[k].stride(0))]
    need = ws(plan.handle, 6, 4, 2, 0)
    work, y = torch.empty(need + 256, dtype=torch.uint8, device="cuda"), torch.empty_like(d["x"])
    call = lambda w=weights, at=work.data_ptr(), n=need, g=None, top=2: L.tgemm_experts_forward(  # noqa: E731
        plan.handle, 6, 4, top, d["x"].data_ptr(), 64, d["e"].data_ptr(), d["w"].data_ptr(), *w, y.data_ptr(), 64, g, None, None, at, n, None)
    assert call() == tg.OK
    assert call(n=need - 1) == tg.ERR_INVALID_ARG and call(at=None) == tg.ERR_INVALID_ARG
    assert call(at=work.data_ptr() + 16) == tg.ERR_ALIGNMENT
    assert call(g=y.data_ptr()) == tg.ERR_INVALID_ARG and call(top=0) == tg.ERR_INVALID_ARG
    assert call(w=[weights[0], 56, *weights[2:]]) == tg.ERR_INVALID_ARG
    assert call(w=[weights[0], 66, *weights[2:]]) == tg.ERR_ALIGNMENT
    assert call(w=[weights[0], 64, weights[2] + 4, *weights[3:]]) == tg.ERR_ALIGNMENT
    plan.close()


@pytest.mark.gpu
def test_no_experts_are_refused_alike(cuda_lib):
    """Whether a plan of these sizes is there already or not."""
    tg, d = cuda_lib, make(27, 6, 4, 2, 56, 88, "bf16")
    d["e"].zero_()
    none = {k: d[k][:0] for k in ("wg", "wu", "wd")}
    for _ in range(2):
        with pytest.raises(ValueError):
            tg.expert_ffn(*args({**d, **none}))
        _, saved = tg.expert_ffn(*args(d), save=True)
        with pytest.raises(ValueError):
            tg.expert_ffn_backward(d["dy"], *args({**d, **none}), saved)
