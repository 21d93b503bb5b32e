"""The calls that feed_forward_operators.md reports on, each twice; run plain, then under ncu."""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import software_pipelined_tiled_02_gb300 as tg  # noqa: E402


def rnd(*shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, device="cuda") * scale).to(dtype)


def norm(rows, width, dtype):
    x, dy, w, b = rnd(rows, width, dtype=dtype), rnd(rows, width, dtype=dtype), rnd(width, dtype=dtype), rnd(width, dtype=dtype)
    _, mean, rstd = tg.layer_norm(x, w, b, stats=True)
    tg.layer_norm_backward(dy, x, mean, rstd, w)


def ffn(tokens, width, hidden, act, dtype, backward):
    x, dy = rnd(tokens, width, dtype=dtype), rnd(tokens, width, dtype=dtype)
    wg, wu, wd = (rnd(*s, dtype=dtype, scale=0.02) for s in ((hidden, width), (hidden, width), (width, hidden)))
    if not backward:
        return tg.gated_ffn(x, wg, wu, wd, activation=act)
    _, saved = tg.gated_ffn(x, wg, wu, wd, activation=act, save=True)
    tg.gated_ffn_backward(dy, x, wg, wu, wd, saved, activation=act)


def cases():
    norm(8192, 4096, torch.bfloat16)
    norm(4000, 3001, torch.float32)
    norm(2000, 16384, torch.float16)
    x = rnd(8192, 4096)
    tg.dropout(x, 0.1, 1, residual=x)
    ffn(1, 4096, 8192, "silu", torch.bfloat16, False)
    ffn(24, 512, 2048, "gelu", torch.float16, False)
    ffn(4096, 2048, 8192, "silu", torch.bfloat16, True)
    ffn(1001, 520, 1400, "gelu", torch.float16, True)


for _ in range(2):
    cases()
torch.cuda.synchronize()
