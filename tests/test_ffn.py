"""The gated feed-forward block on the GPU against its 64-bit definition.

Bounds: a product over K has an fp32 sum of K / 16 tensor-core steps, each off
by at most 2 U of the running sum of absolute values, and 16 terms aligned
within a step: mm(K) = (K / 16 + 16) 2 U times sum |a b|.  Activations carry
64 U relatively and 8 U of |g| absolutely (the error bounds of the fast
exponential and of erff, and the cancellation in 1 + erf).  Every rounding to
the 16-bit type adds u_out, and what was rounded enters the next product.
"""

import os
import subprocess
import sys

import pytest
import torch

import software_pipelined_tiled_02_gb300 as tg_host
from tests import operator_reference as ref
from tests.conftest import ROOT

DT = ref.DTYPES
ACTS = ["silu", "gelu", "relu"]
U = ref.U


def mm(k):
    return (k / 16 + 16) * 2 * U


def make(seed, tokens, width, hidden, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    return {"x": normal(tokens, width), "wg": normal(hidden, width, scale=width ** -0.5),
            "wu": normal(hidden, width, scale=width ** -0.5), "wd": normal(width, hidden, scale=hidden ** -0.5),
            "dy": normal(tokens, width)}


def rounding(v, dt):
    return 1.01 * ref.u_out(dt) * v.abs() + ref.tiny(dt)


def forward_reference(d, act):
    """{name: (value, bound)} of g, u, h and y."""
    dt = d["x"].dtype
    x, wg, wu, wd = (d[k].double() for k in ("x", "wg", "wu", "wd"))
    g, u = x @ wg.T, x @ wu.T
    gb, ub = mm(x.shape[1]) * (x.abs() @ wg.abs().T), mm(x.shape[1]) * (x.abs() @ wu.abs().T)
    a, slope = ref.activation(g, act)
    h = a * u
    ab = slope.abs().clamp(min=1.2) * gb + 64 * U * a.abs() + 8 * U * g.abs()  # |act'| stays below 1.2
    hb = u.abs() * ab + (a.abs() + ab) * ub + rounding(h, dt)
    y = h @ wd.T
    yb = hb @ wd.abs().T + mm(wd.shape[1]) * ((h.abs() + hb) @ wd.abs().T)
    return {"g": (g, gb + rounding(g, dt)), "u": (u, ub + rounding(u, dt)), "h": (h, hb),
            "y": (y, yb + rounding(y.abs() + yb, dt))}


def backward_reference(d, saved, act):
    """{name: (value, bound)} of dx and the weight gradients, from the saved tensors as they are."""
    dt = d["x"].dtype
    x, wg, wu, wd, dy = (d[k].double() for k in ("x", "wg", "wu", "wd", "dy"))
    g, u, h = (t.double() for t in saved)
    tokens, width = x.shape
    a, slope = ref.activation(g, act)
    dh = dy @ wd
    dhb = mm(width) * (dy.abs() @ wd.abs())
    dg, du = dh * u * slope, dh * a
    ab, sb = 64 * U * a.abs() + 8 * U * g.abs(), 64 * U * (1 + g.abs())
    dgb = u.abs() * (slope.abs() * dhb + (dh.abs() + dhb) * sb) + rounding(dg, dt)
    dub = a.abs() * dhb + (dh.abs() + dhb) * ab + rounding(du, dt)
    out = {}
    dx = dg @ wg + du @ wu
    mag = (dg.abs() + dgb) @ wg.abs() + (du.abs() + dub) @ wu.abs()
    out["dx"] = (dx, dgb @ wg.abs() + dub @ wu.abs() + mm(2 * g.shape[1] + 128) * mag)
    for name, left, lb, right in (("dw_gate", dg, dgb, x), ("dw_up", du, dub, x), ("dw_down", dy, dy * 0, h)):
        out[name] = (left.T @ right, lb.abs().T @ right.abs() + mm(tokens) * ((left.abs() + lb).T @ right.abs()))
    return {k: (v, b + rounding(v.abs() + b, dt)) for k, (v, b) in out.items()}


def within(got, want, bound, what):
    assert got.shape == want.shape, what
    off = (got.double() - want).abs()
    ok = off <= bound
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} off, worst error/bound {float((off / bound).max()):.3g}"


def check_forward(tg, d, act, **kw):
    want = forward_reference(d, act)
    y, saved = tg.gated_ffn(d["x"], d["wg"], d["wu"], d["wd"], act, save=True, **kw)
    for name, t in zip("yguh", (y, *saved)):
        within(t, *want[name], name)
    served = tg.gated_ffn(d["x"], d["wg"], d["wu"], d["wd"], act, **kw)
    within(served, *want["y"], "y without save")
    return y, saved


def check_backward(tg, d, saved, act):
    got = tg.gated_ffn_backward(d["dy"], d["x"], d["wg"], d["wu"], d["wd"], saved, act)
    want = backward_reference(d, saved, act)
    for name, t in zip(("dx", "dw_gate", "dw_up", "dw_down"), got):
        within(t, *want[name], name)
    return got


SHAPES = [(1, 8, 8), (3, 8, 24), (5, 64, 64), (8, 72, 200), (9, 128, 256), (16, 264, 520), (17, 512, 1000),
          (31, 136, 2048), (33, 1000, 136), (64, 640, 512), (65, 520, 1400), (127, 256, 264), (129, 96, 1032),
          (256, 256, 256), (257, 264, 520), (700, 328, 648)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(cuda_lib, shape, act, dtype):
    d = make(sum(shape), *shape, dtype)
    _, saved = check_forward(cuda_lib, d, act)
    check_backward(cuda_lib, d, saved, act)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2500, 1032, 2056), (300, 8192, 264), (4100, 136, 4096), (40, 4096, 8192),
                                   (1, 5000, 3000), (4, 1024, 16384), (5003, 136, 128), (3001, 520, 72), (28, 512, 16384),
                                   (200, 168, 8200), (130, 2048, 2056), (641, 96, 3000)])
def test_larger_shapes(cuda_lib, shape):
    """More tiles than CTA pairs, long reductions, many hidden units for few tokens."""
    d = make(7, *shape, "bf16")
    _, saved = check_forward(cuda_lib, d, "silu")
    check_backward(cuda_lib, d, saved, "silu")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 128, 1096), (24, 264, 2112), (40, 520, 1160), (9, 264, 4168), (100, 1096, 264),
                                   (12, 2112, 136), (24, 520, 1608), (513, 72, 1096)])
def test_reductions_that_clusters_share_unevenly(cuda_lib, shape):
    """K blocks that leave a cluster's last CTAs with fewer than the others, or none."""
    d = make(11, *shape, "f16")
    _, saved = check_forward(cuda_lib, d, "gelu")
    check_backward(cuda_lib, d, saved, "gelu")


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", list(range(1, 41)) + [47, 48, 49, 63, 96, 128])
def test_token_counts(cuda_lib, tokens):
    d = make(tokens, tokens, 256, 384, "f16")
    check_forward(cuda_lib, d, "gelu")


def widened(t, pad):
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 7, 40, 300])
def test_strided_rows_and_packed_weights(cuda_lib, tokens):
    """Rows apart from one another with NaN between them; gate and up weights as halves of one matrix."""
    tg = cuda_lib
    d = make(11, tokens, 200, 328, "bf16")
    packed = torch.cat([d["wg"], d["wu"]])
    wide = dict(d, x=widened(d["x"], 8), dy=widened(d["dy"], 24), wd=widened(d["wd"], 16), wg=packed[:328],
                wu=packed[328:])
    y, saved = check_forward(tg, wide, "silu")
    got = check_backward(tg, wide, saved, "silu")
    y0, saved0 = tg.gated_ffn(d["x"], d["wg"], d["wu"], d["wd"], save=True)
    same = tg.gated_ffn_backward(d["dy"], d["x"], d["wg"], d["wu"], d["wd"], saved0)
    for a, b in zip((y, *saved, *got), (y0, *saved0, *same)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_integer_values_are_exact(cuda_lib):
    """relu of small integers: every sum and product is exact in fp32 and in fp16's range, so nothing may differ."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def ints(*shape):
        return torch.randint(-2, 3, shape, generator=gen, device="cuda").half()

    for tokens in (1, 20, 130, 513):
        x, wg, wu, wd, dy = ints(tokens, 24), ints(40, 24), ints(40, 24), ints(24, 40) * 0, ints(tokens, 24)
        wd[:, ::8] = ints(24, 5)
        y, (g, u, h) = cuda_lib.gated_ffn(x, wg, wu, wd, "relu", save=True)
        assert torch.equal(g, (x.double() @ wg.double().T).half()) and torch.equal(u, (x.double() @ wu.double().T).half())
        assert torch.equal(h, (g.double().clamp(min=0) * u.double()).half())
        assert torch.equal(y, (h.double() @ wd.double().T).half())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(cuda_lib, act):
    """The kernels' gradients along random directions against central differences of the 64-bit forward pass."""
    tokens, width, hidden, h = 12, 64, 96, 1e-6
    d = make(13, tokens, width, hidden, "f16")
    _, saved = check_forward(cuda_lib, d, act)
    got = cuda_lib.gated_ffn_backward(d["dy"], d["x"], d["wg"], d["wu"], d["wd"], saved, act)
    want = backward_reference(d, saved, act)
    names = ("x", "wg", "wu", "wd")
    at = {k: d[k].double() for k in names}

    def loss(v):
        a, _ = ref.activation(v["x"] @ v["wg"].T, act)
        return float((d["dy"].double() * ((a * (v["x"] @ v["wu"].T)) @ v["wd"].T)).sum())

    gen = torch.Generator(device="cuda").manual_seed(5)
    for name, grad, key in zip(names, got, ("dx", "dw_gate", "dw_up", "dw_down")):
        v = torch.randn(at[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        slope = (loss(dict(at, **{name: at[name] + h * v})) - loss(dict(at, **{name: at[name] - h * v}))) / (2 * h)
        # g, u and h were rounded to fp16 before the backward pass saw them: each gradient is a sum of products of
        # at most three of them and act', so a few 2^-11 of the sum of absolute values; relu's corner adds none here
        scale = float((want[key][0].abs() * v.abs()).sum())
        tol = float((want[key][1] * v.abs()).sum()) + 8 * 2.0 ** -11 * scale + 1e-4 * (1 + abs(slope))
        assert abs(float((grad.double() * v).sum()) - slope) <= tol, name


@pytest.mark.gpu
def test_no_tokens(cuda_lib):
    d = make(17, 0, 64, 72, "bf16")
    y, saved = cuda_lib.gated_ffn(d["x"], d["wg"], d["wu"], d["wd"], save=True)
    assert y.shape == (0, 64) and saved[0].shape == (0, 72)
    dx, *dw = cuda_lib.gated_ffn_backward(d["dy"], d["x"], d["wg"], d["wu"], d["wd"], saved)
    assert dx.shape == (0, 64) and [tuple(t.shape) for t in dw] == [(72, 64), (72, 64), (64, 72)]
    assert not any(bool(t.any()) for t in dw)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [6, 200])
def test_nan_and_infinity_stay_in_their_token(cuda_lib, tokens):
    tg = cuda_lib
    d = make(19, tokens, 128, 256, "bf16")
    clean = tg.gated_ffn(d["x"], d["wg"], d["wu"], d["wd"])
    x = d["x"].clone()
    x[1, 3], x[4, 127] = float("nan"), float("inf")
    y = tg.gated_ffn(x, d["wg"], d["wu"], d["wd"])
    keep = torch.ones(tokens, dtype=torch.bool, device="cuda")
    keep[[1, 4]] = False
    assert torch.equal(y[keep], clean[keep]) and not y[~keep].isfinite().any()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_extreme_gates(cuda_lib, act):
    """Gates where exp overflows or underflows: the activation's limits, no NaN."""
    gates = torch.tensor([-60000.0, -1000.0, -100.0, -88.5, -20.0, 0.0, 20.0, 88.5, 100.0, 60000.0])
    for tokens in (10, 40):
        x = torch.zeros(tokens, 16, dtype=torch.float16, device="cuda")
        x[:10, 0], x[:, 1] = gates.half().cuda(), 1
        wg, wu, wd = (torch.zeros(s, dtype=torch.float16, device="cuda") for s in ((8, 16), (8, 16), (16, 8)))
        wg[:, 0], wu[:, 1], wd[:, 0] = 1, 0.5, 1
        d = {"x": x, "wg": wg, "wu": wu, "wd": wd, "dy": torch.ones_like(x)}
        _, saved = check_forward(cuda_lib, d, act)
        # The largest gate's du (16 x 60000) leaves fp16's range: it becomes infinite, as documented, and so do its
        # token's dx and its hidden unit's weight gradients.  Everything else keeps its bound.
        a, _ = ref.activation(saved[0], act)
        over = ((d["dy"].double() @ wd.double()) * a).abs() > 65520
        assert int(over.sum()) == 1 and bool(over[9, 0])
        got = cuda_lib.gated_ffn_backward(d["dy"], x, wg, wu, wd, saved, act)
        want = backward_reference(d, saved, act)
        fine = {"dx": ~over.any(1), "dw_gate": torch.ones(8, dtype=torch.bool, device="cuda"), "dw_up": ~over.any(0),
                "dw_down": torch.ones(16, dtype=torch.bool, device="cuda")}
        for (name, keep), t in zip(fine.items(), got):
            value, bound = want[name][0][keep], want[name][1][keep]
            far = value.abs() > 65520 + bound  # the gradient itself leaves fp16's range (x holds 60000)
            assert torch.equal(t[keep].isinf(), far), name
            within(t[keep][~far], value[~far], bound[~far], name)
            assert not t[~keep][:, 1].isfinite().any(), name


@pytest.mark.gpu
def test_same_bits_again_on_another_stream_and_in_a_graph(cuda_lib):
    tg = cuda_lib
    for tokens in (3, 600):
        d = make(23, tokens, 520, 1032, "bf16")
        w = (d["wg"], d["wu"], d["wd"])
        y, saved = tg.gated_ffn(d["x"], *w, save=True)
        want = (y, *saved, *tg.gated_ffn_backward(d["dy"], d["x"], *w, saved))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y2, saved2 = tg.gated_ffn(d["x"], *w, save=True, stream=side)
        got = (y2, *saved2, *tg.gated_ffn_backward(d["dy"], d["x"], *w, saved2, stream=side))
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y3, saved3 = tg.gated_ffn(d["x"], *w, save=True)
            got = (y3, *saved3, *tg.gated_ffn_backward(d["dy"], d["x"], *w, saved3))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
def test_back_to_back_and_from_several_threads(cuda_lib):
    """Calls that follow one another without a wait, each reading what the one before wrote, and calls from four
    threads on their own streams: the bits of calls made one at a time."""
    import threading

    tg = cuda_lib
    shapes = [(5, 256, 512), (70, 256, 512), (400, 256, 512), (3000, 256, 512)]

    def chain(x, w, wait):
        for _ in range(6):
            y, saved = tg.gated_ffn(x, *w, save=True)
            if wait:
                torch.cuda.synchronize()
            dx = tg.gated_ffn_backward(y, x, *w, saved)[0]
            if wait:
                torch.cuda.synchronize()
            x, mean, rstd = tg.layer_norm(tg.dropout(dx, 0.1, 3, 4, residual=x), stats=True)
            if wait:
                torch.cuda.synchronize()
        return x

    data = [make(41 + i, *shape, "bf16") for i, shape in enumerate(shapes)]
    want = [chain(d["x"], (d["wg"], d["wu"], d["wd"]), True) for d in data]
    for d, r in zip(data, want):
        assert torch.equal(chain(d["x"], (d["wg"], d["wu"], d["wd"]), False), r)
    got = [None] * len(data)

    def work(i):
        d, side = data[i], torch.cuda.Stream()
        with torch.cuda.stream(side):
            got[i] = chain(d["x"], (d["wg"], d["wu"], d["wd"]), False)
        side.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_outputs_stay_inside_their_matrices(cuda_lib):
    """The C entry points with guard bands around every output, and the optional outputs left out."""
    tg = cuda_lib
    tokens, D, F = 131, 72, 88
    d = make(29, tokens, D, F, "f16")
    L, plan = tg.load(), tg.GatedFFN(D, F, "f16", "silu")
    shapes = {"y": (tokens, D), "g": (tokens, F), "u": (tokens, F), "h": (tokens, F), "dx": (tokens, D),
              "dwg": (F, D), "dwu": (F, D), "dwd": (D, F), "dg": (tokens, F), "du": (tokens, F)}
    guard = 4096
    room = {k: torch.full((guard + r * c + guard,), 7.0, dtype=torch.float16, device="cuda") for k, (r, c) in shapes.items()}
    out = {k: room[k][guard:-guard].view(shapes[k]) for k in shapes}
    P = {k: t.data_ptr() for k, t in {**d, **out}.items()}
    weights = (P["wg"], D, P["wu"], D, P["wd"], F)
    s = torch.cuda.current_stream().cuda_stream
    assert L.tgemm_ffn_forward(plan.handle, tokens, P["x"], D, *weights, P["y"], D, P["g"], P["u"], P["h"], s) == tg.OK
    head = (plan.handle, tokens, P["dy"], D, P["x"], D, *weights, P["g"], P["u"], P["h"])
    tail = (P["dg"], P["du"], s)
    assert L.tgemm_ffn_backward(*head, P["dx"], D, P["dwg"], P["dwu"], P["dwd"], *tail) == tg.OK
    torch.cuda.synchronize()
    assert plan.status()[0] == tg.OK
    y, saved = tg.gated_ffn(d["x"], d["wg"], d["wu"], d["wd"], save=True)
    grads = tg.gated_ffn_backward(d["dy"], d["x"], d["wg"], d["wu"], d["wd"], saved)
    for k, t in zip(("y", "g", "u", "h", "dx", "dwg", "dwu", "dwd"), (y, *saved, *grads)):
        assert torch.equal(out[k], t), k
        assert bool((room[k][:guard] == 7).all()) and bool((room[k][-guard:] == 7).all()), k
    for left_out in ("dx", "dwg", "dwu", "dwd"):
        for k in ("dx", "dwg", "dwu", "dwd"):
            out[k].fill_(7)
        q = [None if k == left_out else P[k] for k in ("dx", "dwg", "dwu", "dwd")]
        assert L.tgemm_ffn_backward(*head, q[0], D, *q[1:], *tail) == tg.OK
        for k, t in zip(("dx", "dwg", "dwu", "dwd"), grads):
            assert torch.equal(out[k], torch.full_like(t, 7) if k == left_out else t), (left_out, k)
    plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(3000, 128, 4096), (300, 128, 256), (24, 2048, 136)])
def test_watchdog(cuda_lib, shape):
    """A stalled pipeline ends with a status, and the plan works again afterwards: CTA pairs, single CTAs and clusters."""
    tg = cuda_lib
    d = make(31, *shape, "bf16")
    plan = tg.GatedFFN(*shape[1:], "bf16", "silu")
    want = plan.forward(d["x"], d["wg"], d["wu"], d["wd"])
    plan.set_watchdog_ns(20_000_000)
    plan.debug_stall(True)
    plan.forward(d["x"], d["wg"], d["wu"], d["wd"])
    torch.cuda.synchronize()
    assert plan.status()[0] == tg.ERR_TIMEOUT
    plan.debug_stall(False)
    plan.set_watchdog_ns(0)
    assert torch.equal(plan.forward(d["x"], d["wg"], d["wu"], d["wd"]), want)
    torch.cuda.synchronize()
    assert plan.status()[0] == tg.OK
    plan.close()


@pytest.mark.gpu
def test_debug_check_build(cuda_lib):
    """A part of these tests against the build that checks its addresses."""
    if os.environ.get("TGEMM_LIB"):
        pytest.skip("already running against another build")
    from software_pipelined_tiled_02_gb300 import build

    env = dict(os.environ, TGEMM_LIB=build.build(debug=True))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_ffn.py"), "-q", "-x", "-m", "gpu",
                        "-k", "(test_shapes and silu-bf16) or test_strided or test_integer or test_outputs"],
                       cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]


@pytest.mark.gpu
def test_refusals(cuda_lib):
    tg = cuda_lib
    d = make(37, 10, 64, 72, "bf16")
    w = (d["wg"], d["wu"], d["wd"])
    x = d["x"]
    with pytest.raises(tg.TgemmError) as e:
        tg.gated_ffn(x.float(), *(t.float() for t in w))
    assert e.value.code == tg.ERR_UNSUPPORTED_DTYPE
    with pytest.raises(tg.TgemmError) as e:
        tg.gated_ffn(x[:, :60].contiguous(), *w)
    assert e.value.code == tg.ERR_ALIGNMENT
    with pytest.raises(ValueError):
        tg.gated_ffn(x, *w, activation="tanh")
    with pytest.raises(ValueError):
        tg.gated_ffn(x[0], *w)
    with pytest.raises(ValueError):
        tg.gated_ffn(x.cpu(), *w)
    with pytest.raises(ValueError):
        tg.gated_ffn(x, d["wg"], d["wu"].cpu(), d["wd"])
    with pytest.raises(TypeError):
        tg.gated_ffn(x, d["wg"], d["wu"].half(), d["wd"])
    with pytest.raises(ValueError):
        tg.gated_ffn(x, d["wg"], d["wu"][:64], d["wd"])
    with pytest.raises(ValueError):
        tg.gated_ffn(x, d["wg"], d["wu"], d["wd"].t().contiguous().t())
    with pytest.raises(ValueError):
        tg.gated_ffn(x[:1].expand(10, 64), *w)
    for off in (widened(x, 3), widened(torch.cat([x[:, :1], x], 1), 7)[:, 1:65]):  # rows off the 16-byte boundary
        with pytest.raises(tg.TgemmError) as e:
            tg.gated_ffn(off, *w)
        assert e.value.code == tg.ERR_ALIGNMENT
    y, saved = tg.gated_ffn(x, *w, save=True)
    with pytest.raises(ValueError):
        tg.gated_ffn_backward(d["dy"][:5], x, *w, saved)
    with pytest.raises(ValueError):
        tg.gated_ffn_backward(d["dy"], x, *w, (widened(saved[0], 8), *saved[1:]))


def test_validation_without_a_gpu():
    L = tg_host.load()
    v = L.tgemm_ffn_validate
    assert v(4096, 8192, tg_host.BF16, 0) == tg_host.OK
    assert v(8, 8, tg_host.F16, 2) == tg_host.OK
    assert v(64, 64, tg_host.F32, 0) == tg_host.ERR_UNSUPPORTED_DTYPE
    assert v(0, 64, tg_host.F16, 0) == tg_host.ERR_INVALID_ARG
    assert v(64, -8, tg_host.F16, 0) == tg_host.ERR_INVALID_ARG
    assert v(64, (1 << 24) + 8, tg_host.F16, 0) == tg_host.ERR_INVALID_ARG
    assert v(64, 64, tg_host.F16, 3) == tg_host.ERR_INVALID_ARG
    assert v(60, 64, tg_host.F16, 0) == tg_host.ERR_ALIGNMENT
    assert v(64, 100, tg_host.F16, 0) == tg_host.ERR_ALIGNMENT
