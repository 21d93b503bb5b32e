"""The calls that mixture_operators.md reports on, one by its name; run plain, then under ncu:

    python profiles/mixture_calls.py route | route_backward | experts | experts_backward | few | token | product
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import software_pipelined_tiled_02_gb300 as tg  # noqa: E402

gen = torch.Generator(device="cuda").manual_seed(1)


def normal(*shape, scale=0.03):
    return (torch.randn(*shape, device="cuda", generator=gen) * scale).bfloat16()


def route(backward=False):
    """8192 tokens, 8 of 256 experts: sigmoid, bias, 4 of 8 groups; and the gradient of those weights' logits."""
    logits, bias = torch.randn(8192, 256, device="cuda", generator=gen) * 1.5, torch.randn(256, device="cuda", generator=gen) * 0.1
    w, e = tg.route(logits, 8, "sigmoid", bias=bias, groups=8, top_groups=4, group_scores=2)
    if backward:
        tg.route_backward(w, logits, e, "sigmoid")


def experts(tokens, backward=False, save=False):
    """6 of 16 experts of 2048 x 1408."""
    width, hidden, count, top = 2048, 1408, 16, 6
    wg, wu, wd = normal(count, hidden, width), normal(count, hidden, width), normal(count, width, hidden)
    x, dy = normal(tokens, width, scale=1.0), normal(tokens, width, scale=1.0)
    w, e = tg.route(torch.randn(tokens, count, device="cuda", generator=gen), top)
    r = tg.expert_ffn(x, e, w, wg, wu, wd, save=save)
    if backward:
        tg.expert_ffn_backward(dy, x, e, w, wg, wu, wd, r[1])


def product():
    """One token, 16384 x 8192 4-bit weights in groups of 128."""
    packed = torch.randint(0, 256, (16384, 4096), dtype=torch.uint8, device="cuda", generator=gen)
    tg.gemm_w4(normal(1, 8192), packed, normal(16384, 64).abs())


CALLS = {"route": route, "route_backward": lambda: route(True), "experts": lambda: experts(2048, save=True),
         "experts_backward": lambda: experts(2048, True, True), "few": lambda: experts(8), "token": lambda: experts(1), "product": product}

if __name__ == "__main__":
    if len(sys.argv) != 2 or sys.argv[1] not in CALLS:
        raise SystemExit(f"one of {', '.join(CALLS)}")
    CALLS[sys.argv[1]]()
    torch.cuda.synchronize()
