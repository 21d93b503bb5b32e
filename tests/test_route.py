"""Routing of tokens to experts and its gradient against the 64-bit definition."""

import random

import pytest
import torch

from tests import expert_reference as exp
from tests import operator_reference as ref

DT = ref.DTYPES
U = ref.U


def make(seed, tokens, experts, dtype, scale=1.5):
    gen = torch.Generator().manual_seed(seed)
    logits = (torch.randn(tokens, experts, generator=gen) * scale).to(DT[dtype])
    bias = torch.randn(experts, generator=gen) * 0.1
    return logits, bias


def check(tg, logits, top, scoring="softmax", bias=None, **kw):
    w, e = tg.route(logits.cuda(), top, scoring, bias=bias.cuda() if bias is not None else None, **kw)
    assert w.dtype == torch.float32 and e.dtype == torch.int32 and w.shape == e.shape == (len(logits), top)
    want_w, want_e = exp.route(logits, top, scoring, bias, **kw)
    assert torch.equal(e.cpu().long(), want_e)
    off = (w.cpu().double() - want_w).abs()
    assert bool((off <= exp.weight_bound(logits, want_w)).all()), float((off / exp.weight_bound(logits, want_w)).max())
    return w, e


def test_reference_on_a_case_by_hand():
    logits = torch.tensor([[0.0, 1.0, 1.0, -1.0]])
    w, e = exp.route(logits, 2, "sigmoid", bias=torch.tensor([0.5, 0.0, 0.0, 0.0]))
    assert e.tolist() == [[0, 1]]  # 0.5 + 0.5 before 0.731; of the two equal ones the first
    s = [0.5, 1 / (1 + 2.718281828459045 ** -1)]
    assert abs(float(w[0, 0]) - s[0] / sum(s)) < 1e-12
    _, e = exp.route(logits, 1, "softmax", groups=2, top_groups=1, group_scores=2)
    assert e.tolist() == [[1]]


SHAPES = [(1, 1, 1), (1, 2, 2), (3, 7, 1), (32, 32, 4), (5, 33, 6), (64, 64, 8), (17, 100, 3), (9, 128, 8), (33, 129, 2),
          (100, 256, 8), (6, 257, 32), (7, 512, 10), (5, 1000, 32), (4, 1024, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(cuda_lib, shape, scoring, biased, renormalize):
    tokens, experts, top = shape
    for dtype in ("f32", "bf16", "f16"):
        logits, bias = make(sum(shape), tokens, experts, dtype)
        check(cuda_lib, logits, top, scoring, bias if biased else None, renormalize=renormalize, scale=2.5)


GROUPS = [(8, 2, 1, 2), (64, 8, 4, 8), (64, 4, 1, 6), (256, 8, 4, 8), (256, 32, 3, 8), (96, 3, 2, 5), (40, 8, 7, 8), (8, 8, 3, 3),
          (160, 8, 3, 6), (992, 31, 5, 20), (1024, 16, 16, 9)]


@pytest.mark.gpu
@pytest.mark.parametrize("group_scores", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups,top", GROUPS)
def test_groups(cuda_lib, experts, groups, top_groups, top, scoring, biased, group_scores):
    for dtype in ("f32", "bf16"):
        logits, bias = make(experts + groups, 40, experts, dtype)
        check(cuda_lib, logits, top, scoring, bias if biased else None, groups=groups, top_groups=top_groups,
              group_scores=group_scores)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_ties_go_to_the_lowest_index(cuda_lib, scoring, groups, top_groups):
    """Logits and biases of a few values: most keys and most groups are equal."""
    rng = random.Random(3)
    logits = torch.tensor([[rng.choice([-1.0, 0.0, -0.0, 0.5]) for _ in range(72)] for _ in range(60)])
    bias = torch.tensor([rng.choice([0.0, 0.25]) for _ in range(72)])
    for b in (None, torch.zeros(72), bias):
        for group_scores in (1, 2):
            check(cuda_lib, logits, 8, scoring, b, groups=groups, top_groups=top_groups, group_scores=group_scores)
    check(cuda_lib, torch.zeros(5, 72), 8, scoring, torch.zeros(72), groups=groups, top_groups=top_groups, group_scores=2)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_keys_nearer_than_fp32_tells_apart(cuda_lib, scoring):
    """Every bias fills its expert's score up to one value, to fp32's rounding: keys differ by some 1e-8, and the order
    is that of 64 bits."""
    gen = torch.Generator().manual_seed(11)
    row = torch.randn(96, generator=gen)
    logits = row.repeat(8, 1)
    logits[1:] += torch.randn(7, 96, generator=gen) * 1e-7
    bias = (0.75 - exp.scores(row[None], scoring)[0]).float()
    for groups, top_groups in ((1, 1), (4, 2), (12, 5)):
        for group_scores in (1, 2):
            check(cuda_lib, logits, 8, scoring, bias, groups=groups, top_groups=top_groups, group_scores=group_scores)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_keys_of_unlike_errors_a_few_roundings_apart(cuda_lib, scoring):
    """Keys some 1e-7 apart, half of them from scores that fp32 hardly knows and half from biases alone: one of the first
    kind may stand two places from where its fp32 key puts it."""
    gen = torch.Generator().manual_seed(13)
    for trial in range(20):
        row = torch.where(torch.rand(64, generator=gen) < 0.5, torch.full((64,), -18.0), 2.0 + torch.rand(64, generator=gen))
        want = 0.75 + torch.randperm(64, generator=gen) * 2.0 ** -24
        bias = (want.double() - exp.scores(row[None], scoring)[0]).float()
        check(cuda_lib, row.repeat(3, 1), 9, scoring, bias)


@pytest.mark.gpu
def test_saturated_sigmoids_keep_the_order_of_logits(cuda_lib):
    logits = torch.arange(20.0, 116.0).repeat(3, 1)
    check(cuda_lib, logits, 5, "sigmoid")
    check(cuda_lib, -logits, 5, "sigmoid")  # scores down to 1e-50: the quotients are still right


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_experts_and_empty_rows(cuda_lib, scoring, renormalize, biased):
    logits, bias = make(5, 6, 40, "f32")
    logits[0, 5:] = -float("inf")   # as many as are chosen
    logits[1, 2:] = -float("inf")   # fewer
    logits[2] = -float("inf")       # none
    logits[3, ::2] = torch.finfo(torch.float32).min
    w, e = check(cuda_lib, logits, 5, scoring, bias if biased else None, renormalize=renormalize)
    assert not w[2].any() and not w.isnan().any()
    if biased:  # an expert that is switched off through its bias
        bias[7] = -float("inf")
        check(cuda_lib, logits, 5, scoring, bias, renormalize=renormalize)


@pytest.mark.gpu
def test_nan_and_infinity(cuda_lib):
    tg = cuda_lib
    logits = torch.zeros(3, 40)
    logits[0, 7] = float("nan")
    logits[1, 9] = float("inf")
    for scoring in ("softmax", "sigmoid"):
        for bias in (None, torch.linspace(0, 1, 40).cuda()):
            w, e = tg.route(logits.cuda(), 3, scoring, bias=bias)
            assert all(len(set(r)) == 3 and 0 <= min(r) and max(r) < 40 for r in e.tolist())
            if bias is None or scoring == "sigmoid":
                assert e[0, 0] == 7
            assert bool(w[0].isnan().all()) and not w[2].isnan().any()
    w, e = tg.route(logits.cuda(), 3, "sigmoid")
    assert e[1].tolist() == [9, 0, 1] and torch.equal(w[1].cpu(), torch.tensor([1.0, 0.5, 0.5]) / 2)


@pytest.mark.gpu
def test_many_rows_strides_and_streams(cuda_lib):
    tg = cuda_lib
    logits, bias = make(9, 5000, 60, "bf16")
    want = check(tg, logits, 6, "sigmoid", bias)
    wide = torch.full((5000, 77), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:63] = logits.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tg.route(wide[:, 3:63], 6, "sigmoid", bias=bias.cuda(), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    empty = tg.route(torch.empty(0, 60, device="cuda"), 6)
    assert empty[0].shape == empty[1].shape == (0, 6)
    assert tg.route_backward(empty[0], torch.empty(0, 60, device="cuda"), empty[1]).shape == (0, 60)


INF, MOST = float("inf"), torch.finfo(torch.float32).max


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [INF, -INF, MOST, -MOST])
@pytest.mark.parametrize("experts,top", [(40, 3), (7, 2), (256, 8), (1000, 5)])
def test_biases_that_force_or_forbid(cuda_lib, experts, top, value, scoring):
    """One expert, as many as are chosen, one fewer and one more, all but one, all."""
    logits, bias = make(experts + top, 9, experts, "f32")
    logits[3:6] = logits[3:6].round()  # equal scores among them
    for count in (1, top - 1, top, top + 1, experts - top, experts - 1, experts):
        some = bias.clone()
        some[torch.randperm(experts, generator=torch.Generator().manual_seed(count))[:count]] = value
        check(cuda_lib, logits, top, scoring, some)
        check(cuda_lib, logits.round(), top, scoring, torch.where(some == value, some, torch.zeros(())))


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_infinite_and_largest_biases_together(cuda_lib, scoring):
    rng = random.Random(17)
    logits, _ = make(17, 40, 72, "f32")
    for trial in range(20):
        bias = torch.tensor([rng.choice([0.0, 0.1, INF, -INF, MOST, -MOST, MOST / 2, 1e30, -1e7]) for _ in range(72)])
        check(cuda_lib, logits, rng.choice([1, 2, 8, 20, 32]), scoring, bias)


INFINITE_GROUPS = [(64, 8, 4, 8), (64, 4, 2, 6), (256, 8, 4, 8), (96, 3, 2, 5), (40, 8, 7, 8), (8, 8, 3, 3), (992, 31, 5, 20)]


@pytest.mark.gpu
@pytest.mark.parametrize("group_scores", [1, 2])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("experts,groups,top_groups,top", INFINITE_GROUPS)
def test_groups_that_infinite_biases_force_or_forbid(cuda_lib, experts, groups, top_groups, top, value, scoring, group_scores):
    """One or two experts of some groups, all but one, and whole groups: in fewer, as many and more groups than are chosen."""
    logits, bias = make(experts + top, 9, experts, "f32")
    size = experts // groups
    for count in {1, top_groups - 1, top_groups, top_groups + 1, groups - 1, groups} - {0}:
        at = torch.randperm(groups, generator=torch.Generator().manual_seed(count))[:count]
        for each in {1, min(2, size), max(1, size - 1), size}:
            some = bias.reshape(groups, size).clone()
            some[at, :each] = value
            some = some.flatten()
            check(cuda_lib, logits, top, scoring, some, groups=groups, top_groups=top_groups, group_scores=group_scores)


@pytest.mark.gpu
@pytest.mark.parametrize("group_scores", [1, 2])
@pytest.mark.parametrize("from_bias", [False, True])
def test_nan_leaves_the_other_groups_in_exact_order(cuda_lib, from_bias, group_scores):
    """Groups whose scores differ by less than fp32 tells apart, beside one with a NaN (of a sigmoid's logit, or of the bias)."""
    gen = torch.Generator().manual_seed(19)
    logits = torch.randn(96, generator=gen).repeat(30, 1)
    logits[1:] += torch.randn(29, 96, generator=gen) * 1e-7
    bias = (0.75 - exp.scores(logits[:1], "sigmoid")[0]).float()
    forced = bias.clone()
    forced[70] = INF  # ranks its expert and its group as NaN does
    clean = logits.clone()
    if from_bias:
        bias[70] = float("nan")
    else:
        logits[:, 70] = float("nan")
    for groups, top_groups in ((4, 2), (12, 5), (24, 3)):
        _, want = exp.route(clean, 6, "sigmoid", forced, groups=groups, top_groups=top_groups, group_scores=group_scores)
        _, got = cuda_lib.route(logits.cuda(), 6, "sigmoid", bias=bias.cuda(), groups=groups, top_groups=top_groups,
                                group_scores=group_scores)
        assert torch.equal(got.cpu().long(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("group_scores", [1, 2])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups,top", INFINITE_GROUPS)
def test_groups_with_biases_as_large_as_there_are(cuda_lib, experts, groups, top_groups, top, scoring, group_scores):
    """Two of them make a sum that fp32 does not hold, and that stays behind a group that is forced, before one that is
    forbidden."""
    logits, bias = make(experts + top, 9, experts, "f32")
    size, rng = experts // groups, random.Random(23)
    for trial in range(12):
        some = bias.reshape(groups, size).clone()
        for g in range(groups):
            each = rng.choice([0, 1, min(2, size), size])
            some[g, :each] = rng.choice([MOST, -MOST, MOST / 2, INF, -INF])
        some = some.flatten()
        check(cuda_lib, logits, top, scoring, some, groups=groups, top_groups=top_groups, group_scores=group_scores)


def fastest(call, passes=20):
    """The shortest of some passes of ten calls, in us a call."""
    graph = torch.cuda.CUDAGraph()
    call()
    with torch.cuda.graph(graph):
        for _ in range(10):
            call()
    times = []
    for _ in range(passes):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        graph.replay()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end) * 100)
    return min(times)


@pytest.mark.gpu
@pytest.mark.parametrize("group_scores", [1, 2])
@pytest.mark.parametrize("value", [-INF, -MOST])
def test_a_group_switched_off_does_not_slow_the_others(cuda_lib, value, group_scores):
    """Every token went through 64 bits, at several times the cost."""
    logits, bias = (t.cuda() for t in make(29, 8192, 256, "f32"))
    off, most = bias.clone(), bias.clone()
    off[96:128] = value
    most[96:127] = value  # all but one
    kw = {"bias": bias, "groups": 8, "top_groups": 4, "group_scores": group_scores}
    usual = fastest(lambda: cuda_lib.route(logits, 8, "sigmoid", **kw))
    for masked in (off, most):
        assert fastest(lambda: cuda_lib.route(logits, 8, "sigmoid", **{**kw, "bias": masked})) < 1.6 * usual


@pytest.mark.gpu
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 4)])
def test_masked_rows_are_not_slower(cuda_lib, groups, top_groups):
    """Rows of -inf, as those of padding, have exact keys: their biases."""
    logits, bias = make(37, 8192, 256, "f32")
    masked = torch.full_like(logits, -INF)
    check(cuda_lib, masked[:3], 8, "softmax", bias, groups=groups, top_groups=top_groups, group_scores=2)
    logits, masked, bias = logits.cuda(), masked.cuda(), bias.cuda()
    kw = {"bias": bias, "groups": groups, "top_groups": top_groups, "group_scores": 2}
    usual = fastest(lambda: cuda_lib.route(logits, 8, "softmax", **kw))
    assert fastest(lambda: cuda_lib.route(masked, 8, "softmax", **kw)) < 1.6 * usual


def test_bound_of_a_sigmoid_key():
    """1 / (1 + exp2(-l log2 e)) as the kernel forms it, with exp2 and the reciprocal off by what the hardware may be."""
    l = torch.linspace(-90.0, 90.0, 400001)
    for exp2_off in (-2.0 ** -22, 0.0, 2.0 ** -22):
        for rcp_off in (-2.0 ** -23, 2.0 ** -23):
            e = (torch.exp2((-l * 1.44269504088896341).double()) * (1 + exp2_off)).float()
            s = (1 + rcp_off) / (1.0 + e).double()
            off = (s - torch.sigmoid(l.double())).abs()
            assert float(off.max()) < 8 * U and float((off / torch.sigmoid(l.double())).max()) > 8 * U


# ------------------------------------------------------------------ the gradient

def check_backward(tg, dw, logits, chosen, scoring, renormalize, scale):
    got = tg.route_backward(dw.cuda(), logits.cuda(), chosen.int().cuda(), scoring, renormalize=renormalize, scale=scale)
    assert got.shape == logits.shape and got.dtype == logits.dtype
    n = logits.shape[1]
    want, mag = exp.route_backward(dw, logits, torch.where((chosen < 0) | (chosen >= n), torch.full_like(chosen, -1), chosen),
                                   scoring, renormalize, scale)
    spread = torch.nan_to_num(logits.double(), neginf=0.0).abs().amax(1, keepdim=True) * 2
    # each share and slope as a weight's bound, the sums over the choices 40 U of what meets, and the output's rounding
    bound = mag * U * (160 + 12 * spread) + 1.01 * ref.u_out(logits.dtype) * want.abs() + ref.tiny(logits.dtype) + 2.0 ** -120
    off = (got.cpu().double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradient(cuda_lib, shape, scoring, renormalize):
    tokens, experts, top = shape
    for dtype in ("f32", "bf16", "f16"):
        logits, _ = make(sum(shape) + 1, tokens, experts, dtype)
        chosen = exp.route(logits, top)[1]
        dw = torch.randn(tokens, top, generator=torch.Generator().manual_seed(1))
        check_backward(cuda_lib, dw, logits, chosen, scoring, renormalize, 2.5)


@pytest.mark.gpu
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_of_odd_choices(cuda_lib, scoring, renormalize):
    """Entries out of range, the same expert twice, masked logits, an empty row."""
    logits, _ = make(21, 6, 45, "f32")
    chosen = exp.route(logits, 4)[1]
    chosen[0, 1], chosen[1, 3], chosen[2] = -1, 45, torch.tensor([7, 7, 3, 7])
    chosen[3] = -5
    logits[4, chosen[4, 2]] = -float("inf")
    logits[5] = -float("inf")
    dw = torch.randn(6, 4, generator=torch.Generator().manual_seed(2))
    got = check_backward(cuda_lib, dw, logits, chosen, scoring, renormalize, 1.0)
    assert not got[5].any()


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_formula_against_differences(scoring, renormalize):
    logits, _ = make(31, 3, 12, "f32")
    logits = logits.double()
    chosen = exp.route(logits, 4)[1]
    dw = torch.randn(3, 4, generator=torch.Generator().manual_seed(3)).double()
    got, _ = exp.route_backward(dw, logits, chosen, scoring, renormalize, 1.5)
    step = 1e-5
    for e in range(12):
        up, down = logits.clone(), logits.clone()
        up[:, e] += step
        down[:, e] -= step
        d = (exp.weights_of(up, chosen, scoring, renormalize, 1.5) - exp.weights_of(down, chosen, scoring, renormalize, 1.5)) / (2 * step)
        assert torch.allclose((d * dw).sum(1), got[:, e], rtol=1e-6, atol=1e-8)


@pytest.mark.gpu
def test_captured(cuda_lib):
    """Replays follow their inputs."""
    tg = cuda_lib
    logits, bias = (t.cuda() for t in make(41, 300, 96, "f32"))
    graph = torch.cuda.CUDAGraph()
    tg.route(logits, 4, "sigmoid", bias=bias)
    with torch.cuda.graph(graph):
        w, e = tg.route(logits, 4, "sigmoid", bias=bias)
        dl = tg.route_backward(w, logits, e, "sigmoid")
    for seed in (1, 2):
        logits.copy_(make(seed, 300, 96, "f32")[0])
        graph.replay()
        w2, e2 = tg.route(logits, 4, "sigmoid", bias=bias)
        assert torch.equal(w, w2) and torch.equal(e, e2) and torch.equal(dl, tg.route_backward(w2, logits, e2, "sigmoid"))


def test_refusals_without_a_gpu():
    import software_pipelined_tiled_02_gb300 as tg

    with pytest.raises(ValueError, match="CUDA tensor"):
        tg.route(torch.zeros(2, 4), 1)
    with pytest.raises(TypeError):
        tg.route([1.0], 1)
    L = tg.load()
    call = lambda **k: L.tgemm_route(*{"t": 4, "e": 8, "top": 2, "dt": tg.F32, "l": None, "ld": 8, "b": None, "s": 0, "g": 1,  # noqa: E731
                                       "tg": 1, "gs": 1, "r": 1, "sc": 1.0, "w": None, "c": None, "st": None, **k}.values())
    assert call(dt=7) == tg.ERR_UNSUPPORTED_DTYPE
    for bad in ({"t": -1}, {"t": 1 << 31}, {"e": 0}, {"e": 1025}, {"top": 0}, {"top": 9}, {"s": 2}, {"g": 3}, {"g": 0}, {"tg": 2},
                {"tg": 0}, {"gs": 0}, {"gs": 3}, {"g": 8, "tg": 1, "top": 2}, {"e": 40, "top": 33}):
        assert call(**bad) == tg.ERR_INVALID_ARG, bad
    assert L.tgemm_route_backward(4, 8, 9, tg.F32, None, None, 8, None, 0, 1, 1.0, None, None) == tg.ERR_INVALID_ARG
    assert L.tgemm_route_backward(4, 8, 2, 5, None, None, 8, None, 0, 1, 1.0, None, None) == tg.ERR_UNSUPPORTED_DTYPE


@pytest.mark.gpu
def test_refusals(cuda_lib):
    tg = cuda_lib
    x = torch.randn(4, 8, device="cuda")
    w, e = tg.route(x, 2)
    for bad in ({"top_k": 0}, {"top_k": 9}, {"top_k": 2, "groups": 3}, {"top_k": 2, "groups": 8, "top_groups": 1},
                {"top_k": 2, "groups": 4, "top_groups": 5}, {"top_k": 2, "group_scores": 3}, {"top_k": 2, "scoring": "tanh"},
                {"top_k": 2, "bias": torch.zeros(7, device="cuda")}, {"top_k": 2, "bias": torch.zeros(8)}, {"top_k": 1 << 40}):
        with pytest.raises(ValueError):
            tg.route(x, **bad)
    for bad in (x.double(), x.long()):
        with pytest.raises(TypeError):
            tg.route(bad, 2)
    with pytest.raises(TypeError):
        tg.route(x, 2, bias=torch.zeros(8, device="cuda").half())
    with pytest.raises(TypeError):
        tg.route(x, 2.5)
    for bad in (x.t(), x[0], torch.zeros(2, 1025, device="cuda"), torch.zeros(2, 0, device="cuda")):
        with pytest.raises(ValueError):
            tg.route(bad, 1)
    with pytest.raises(TypeError):
        tg.route_backward(w, x, e.long())
    with pytest.raises(TypeError):
        tg.route_backward(w.half(), x, e)
    for bad in ((w[:2], x, e), (w, x, e[:, :1]), (w, x[:, :1], e), (w.t(), x, e), (w, x, e.cpu())):
        with pytest.raises(ValueError):
            tg.route_backward(*bad)
    L, p = tg.load(), x.data_ptr()
    assert L.tgemm_route(4, 8, 2, tg.F32, p, 7, None, 0, 1, 1, 1, 1, 1.0, w.data_ptr(), e.data_ptr(), None) == tg.ERR_INVALID_ARG
    assert L.tgemm_route(4, 8, 2, tg.F32, p + 2, 8, None, 0, 1, 1, 1, 1, 1.0, w.data_ptr(), e.data_ptr(), None) == tg.ERR_ALIGNMENT
    assert L.tgemm_route(4, 8, 2, tg.F32, None, 8, None, 0, 1, 1, 1, 1, 1.0, w.data_ptr(), e.data_ptr(), None) == tg.ERR_INVALID_ARG
