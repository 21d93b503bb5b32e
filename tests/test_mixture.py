"""The mixture-of-experts operators together: as examples/mixture_of_experts.py runs
them, under capture from a process's first call on, side by side on two streams, and
with kernels that give up."""

import importlib.util
import os
import random
import subprocess
import sys

import pytest
import torch

from tests import expert_reference as exp
from tests import test_experts
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("mixture_of_experts", os.path.join(ROOT, "examples", "mixture_of_experts.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_runs(cuda_lib, example):
    teacher = example.Block(256, 128, 8, 2, seed=7).eval()
    block = example.Block(256, 128, 8, 2)
    losses = example.train(block, teacher, 1000, 4)
    assert len(losses) == 4 and all(v == v and v < float("inf") for v in losses)
    assert int(block.load.sum()) == 2000 and bool(block.bias.any())


def test_gradients_of_the_whole_block(cuda_lib, example):
    """Against torch's autograd in 64 bits on the same values and choices.  A gradient passes at most a dozen roundings to
    bf16 on its way, each 2^-8 at most and independent, so 12 x 2^-8 bounds its relative error in norm."""
    tokens, width, hidden, experts, top = 300, 128, 264, 8, 3
    block = example.Block(width, hidden, experts, top, activation="gelu", seed=5)
    with torch.no_grad():
        block.norm_w.add_(0.1 * torch.randn(width, device="cuda"))
        block.norm_b.add_(0.1 * torch.randn(width, device="cuda"))
        block.bias.add_(0.05 * torch.randn(experts, device="cuda"))
    x = torch.randn(tokens, width, device="cuda").bfloat16().requires_grad_()
    dout = torch.randn(tokens, width, device="cuda").bfloat16()
    out, chosen = example.MixtureOfExperts.apply(x, block.norm_w, block.norm_b, block.router, block.w_gate, block.w_up, block.w_down,
                                                 block.bias, top, "gelu")
    out.backward(dout)

    names = ("norm_w", "norm_b", "router", "w_gate", "w_up", "w_down")
    d = {name: getattr(block, name).detach().double().requires_grad_() for name in names}
    xd = x.detach().double().requires_grad_()
    n = torch.nn.functional.layer_norm(xd, (width,), d["norm_w"], d["norm_b"])
    s = torch.sigmoid(n @ d["router"].T).gather(1, chosen.long())
    w = s / s.sum(1, keepdim=True)
    y = torch.zeros(tokens, width, dtype=torch.float64, device="cuda")
    for e in range(experts):
        t, j = (chosen == e).nonzero(as_tuple=True)
        h = torch.nn.functional.gelu(n[t] @ d["w_gate"][e].T) * (n[t] @ d["w_up"][e].T)
        y = y.index_add(0, t, w[t, j][:, None] * (h @ d["w_down"][e].T))
    want = xd + y
    want.backward(dout.double())
    pairs = [("out", out, want), ("x", x.grad, xd.grad)] + [(k, getattr(block, k).grad, d[k].grad) for k in names]
    for name, got, exact in pairs:
        off = float((got.double() - exact).norm() / exact.norm())
        assert off < 12 * 2.0 ** -8, f"{name}: {off:.3g}"


def test_serving_with_4_bit_experts(cuda_lib, example):
    """Against the same block in 64 bits with the rounded weights: a few roundings to bf16."""
    width, hidden, experts, top = 256, 384, 12, 3
    block = example.Block(width, hidden, experts, top, seed=3).eval()
    packed = [example.quantize(w.detach()) for w in (block.w_gate, block.w_up, block.w_down)]
    x = torch.randn(5, width, device="cuda").bfloat16()
    with torch.no_grad():
        got = block.served(x, packed)
        n = cuda_lib.layer_norm(x, block.norm_w, block.norm_b)
        weights, chosen = block.route(n)
    wg, wu, wd = (exp.unpack_w4(*p) for p in packed)
    e = chosen.long()
    nd = n.double()[:, None, :, None]
    h = torch.nn.functional.silu(wg[e] @ nd) * (wu[e] @ nd)
    y = ((wd[e] @ h)[..., 0] * weights.double()[..., None]).sum(1)
    off = float(((got - x).double() - y).norm() / y.norm())
    assert off < 4 * 2.0 ** -8 * (1 + float(x.norm() / y.norm())), off


FIRST_CALLS = """
import torch
import software_pipelined_tiled_02_gb300 as tg

gen = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: (torch.randn(*s, device="cuda", generator=gen) * 0.1).bfloat16()
x, wg, wu, wd, dy = r({tokens}, 64), r(6, 72, 64), r(6, 72, 64), r(6, 64, 72), r({tokens}, 64)
logits = torch.randn({tokens}, 6, device="cuda", generator=gen)
packed = torch.randint(0, 256, (6, 40, 32), dtype=torch.uint8, device="cuda")
scales = r(6, 40, 2).abs()
torch.cuda.synchronize()

def step():
    w, e = tg.route(logits, 2, "sigmoid", bias=torch.zeros(6, device="cuda"))
    y, saved = tg.expert_ffn(x, e, w, wg, wu, wd, save=True)
    dx, dw, *rest = tg.expert_ffn_backward(dy, x, e, w, wg, wu, wd, saved)
    return [w, e, y, *saved, dx, dw, *rest, tg.route_backward(dw, logits, e, "sigmoid"), tg.expert_ffn(x, e, w, wg, wu, wd),
            tg.gemm_w4(x, packed, scales, experts=e)]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("same")
"""


@pytest.mark.parametrize("tokens", [3, 300])
def test_a_process_may_begin_with_a_capture(cuda_lib, tokens):
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(tokens=tokens)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("tokens", [4, 400])
def test_two_streams_at_once(cuda_lib, tokens):
    """Steps of two inputs on two streams, call by call in turn, and of one input on both."""
    tg = cuda_lib
    a, b = (test_experts.make(seed, tokens, 9, 2, 136, 264, "bf16") for seed in (31, 32))

    def forward(d, stream):
        y, saved = tg.expert_ffn(*test_experts.args(d), save=True, stream=stream)
        return (y, tg.expert_ffn(*test_experts.args(d), stream=stream), *saved,
                *tg.expert_ffn_backward(d["dy"], *test_experts.args(d), saved, stream=stream))

    want = [forward(d, None) for d in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[forward(d, s) for d, s in zip(order, streams)] for order in ([a, b], [b, a], [a, a]) for _ in range(4)]
    torch.cuda.synchronize()
    for i, pair in enumerate(got):
        first, second = ((0, 1), (1, 0), (0, 0))[i // 4]
        for result, w in zip(pair, (want[first], want[second])):
            assert all(torch.equal(p, q) for p, q in zip(result, w))


def test_two_graphs_replayed_in_turn(cuda_lib):
    tg = cuda_lib
    graphs = []
    for seed, tokens in ((41, 200), (42, 900)):
        d = test_experts.make(seed, tokens, 7, 2, 136, 264, "f16")
        y, saved = tg.expert_ffn(*test_experts.args(d), save=True)
        want = (y, *tg.expert_ffn_backward(d["dy"], *test_experts.args(d), saved))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, saved = tg.expert_ffn(*test_experts.args(d), save=True)
            got = (y, *tg.expert_ffn_backward(d["dy"], *test_experts.args(d), saved))
        graphs.append((graph, got, want, d, saved))
    for _ in range(3):
        for graph, *_ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, got, want, *_ in graphs:
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_a_kernel_that_gives_up_is_reported(cuda_lib):
    from software_pipelined_tiled_02_gb300 import operators

    tg, d = cuda_lib, test_experts.make(51, 300, 5, 2, 232, 440, "bf16")
    want, saved = tg.expert_ffn(*test_experts.args(d), save=True)
    grads = tg.expert_ffn_backward(d["dy"], *test_experts.args(d), saved)
    torch.cuda.synchronize()
    assert tg.gated_ffn_status()[0] == tg.OK
    plan = operators._ffn_plans[232, 440, torch.bfloat16, "silu", 0]
    plan.set_watchdog_ns(20_000_000)
    plan.debug_stall(True)
    for call in (lambda: tg.expert_ffn(*test_experts.args(d), save=True),
                 lambda: tg.expert_ffn_backward(d["dy"], *test_experts.args(d), saved)):
        call()
        torch.cuda.synchronize()
        code, detail = tg.gated_ffn_status()
        assert code == tg.ERR_TIMEOUT and detail[0] == tg.ERR_TIMEOUT
    plan.debug_stall(False)
    plan.set_watchdog_ns(0)
    assert torch.equal(tg.expert_ffn(*test_experts.args(d)), want)
    assert all(torch.equal(a, b) for a, b in zip(tg.expert_ffn_backward(d["dy"], *test_experts.args(d), saved), grads))
    torch.cuda.synchronize()
    assert tg.gated_ffn_status()[0] == tg.OK


# ------------------------------------------------------------------ seeded sizes

CASES = int(os.environ.get("OPERATOR_SWEEP_CASES", "40"))
SEED = int(os.environ.get("OPERATOR_SWEEP_SEED", "20250"))


def log_int(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def route_case(tg, rng):
    from tests import test_route

    groups = rng.choice([1, 1, 2, 3, 8, 16])
    experts = groups * log_int(rng, 1, 1024 // groups)
    top_groups = rng.randint(1, groups)
    top = rng.randint(1, min(32, experts // groups * top_groups))
    logits, bias = test_route.make(rng.randrange(1 << 30), log_int(rng, 1, 60), experts, rng.choice(["f32", "bf16", "f16"]),
                                   scale=rng.choice([0.01, 1.5, 6.0]))
    kw = {"renormalize": rng.random() < 0.6}
    scoring = rng.choice(["softmax", "sigmoid"])
    w, e = test_route.check(tg, logits, top, scoring, bias if rng.random() < 0.6 else None, groups=groups, top_groups=top_groups,
                            group_scores=rng.choice([1, 2]), scale=rng.choice([1.0, 2.5]), **kw)
    test_route.check_backward(tg, torch.randn(w.shape, generator=torch.Generator().manual_seed(1)), logits, e.cpu().long(), scoring,
                              kw["renormalize"], 2.5)


def experts_case(tg, rng):
    while True:
        tokens, experts, width, hidden = log_int(rng, 1, 3000), log_int(rng, 1, 200), 8 * log_int(rng, 1, 200), 8 * log_int(rng, 1, 200)
        top = rng.randint(1, min(8, experts))
        if tokens * top * width * hidden < 1 << 32 and experts * width * hidden < 1 << 28:
            break
    d = test_experts.make(rng.randrange(1 << 30), tokens, experts, top, width, hidden, rng.choice(["bf16", "f16"]),
                          invalid=rng.random() < 0.3)
    act = rng.choice(test_experts.ACTS)
    _, saved = test_experts.check_forward(tg, d, act)
    test_experts.check_backward(tg, d, saved, act)


def w4_case(tg, rng):
    from tests import test_w4

    group = 32 * log_int(rng, 1, 12)
    dtype = rng.choice(["bf16", "f16"])
    rows, width, tokens = log_int(rng, 1, 2000), group * log_int(rng, 1, 30), log_int(rng, 1, 80)
    packed, scales, z = test_w4.make(rng.randrange(1 << 30), rows, width, group, dtype, rng.random() < 0.5,
                                     scale_dtype=rng.choice([None, torch.float32]))
    x = test_w4.rows_of(rng.randrange(1 << 30), tokens, width, dtype=dtype)
    test_w4.within(tg.gemm_w4(x, packed, scales, z), x, exp.unpack_w4(packed, scales, z), group, f"{rows} x {width}, {tokens}")


@pytest.mark.parametrize("case", range(CASES))
def test_sweep(cuda_lib, case):
    rng = random.Random(SEED + case)
    (route_case, experts_case, w4_case)[case % 3](cuda_lib, rng)
