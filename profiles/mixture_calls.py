"""One call of each mixture-of-experts operator at a size whose counters are worth reading: inputs larger than L2 where
the operator streams, a few GB on the device.  Run it alone, or under ncu."""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import software_pipelined_tiled_02_gb300 as tg  # noqa: E402


def main():
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, scale=0.03):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).bfloat16()

    # 8192 tokens, 8 of 256 experts: sigmoid, bias, 4 of 8 groups; and the gradient
    logits, bias = torch.randn(8192, 256, device="cuda", generator=gen) * 1.5, torch.randn(256, device="cuda", generator=gen) * 0.1
    w, e = tg.route(logits, 8, "sigmoid", bias=bias, groups=8, top_groups=4, group_scores=2)
    tg.route_backward(w, logits, e, "sigmoid")
    # 2048 tokens, 6 of 16 experts of 2048 x 1408: forward and backward; then one token
    tokens, experts, top, width, hidden = 2048, 16, 6, 2048, 1408
    wg, wu, wd = normal(experts, hidden, width), normal(experts, hidden, width), normal(experts, width, hidden)
    x, dy = normal(tokens, width, scale=1.0), normal(tokens, width, scale=1.0)
    w, e = tg.route(torch.randn(tokens, experts, device="cuda", generator=gen), top)
    y, saved = tg.expert_ffn(x, e, w, wg, wu, wd, save=True)
    tg.expert_ffn_backward(dy, x, e, w, wg, wu, wd, saved)
    tg.expert_ffn(x[:1], e[:1], w[:1], wg, wu, wd)
    # one token, 16384 x 8192 4-bit weights in groups of 128
    packed = torch.randint(0, 256, (16384, 4096), dtype=torch.uint8, device="cuda", generator=gen)
    tg.gemm_w4(normal(1, 8192), packed, normal(16384, 64).abs())
    torch.cuda.synchronize()


if __name__ == "__main__":
    main()
