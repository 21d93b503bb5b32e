"""Seeded random shapes, types, strides and alignments through the feed-forward
operators, each against its 64-bit definition with its derived bound.

OPERATOR_SWEEP_CASES and OPERATOR_SWEEP_SEED ask for more, and for others.
"""

import os
import random

import pytest
import torch

from tests import operator_reference as ref
from tests import test_ffn, test_norm

pytestmark = pytest.mark.gpu

CASES = int(os.environ.get("OPERATOR_SWEEP_CASES", "120"))
SEED = int(os.environ.get("OPERATOR_SWEEP_SEED", "20240"))


def log_int(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def placed(rng, t):
    """t in rows that are apart, off the 16-byte boundary, or as it is; NaN around it."""
    how = rng.choice(["plain", "plain", "apart", "off"])
    if how == "plain" or t.shape[0] == 0:
        return t
    left, right = (0, rng.choice([8, 3, 16])) if how == "apart" else (rng.choice([1, 4, 8]), rng.choice([0, 5, 7]))
    wide = torch.full((t.shape[0], left + t.shape[1] + right), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[:, left:left + t.shape[1]]
    view.copy_(t)
    return view


def norm_case(tg, rng):
    width = log_int(rng, 1, 20000)
    rows = min(log_int(rng, 1, 20000), max(1, (1 << 22) // width))
    dt = ref.DTYPES[rng.choice(["bf16", "f16", "f32"])]
    wt = rng.choice([dt, torch.float32])
    seed = rng.randrange(1 << 30)
    x, dy = test_norm.rows_of(seed, rows, width, dt), test_norm.rows_of(seed + 1, rows, width, dt, shift=0.0)
    w = test_norm.rows_of(seed + 2, 1, width, wt, shift=1.0)[0] if rng.random() < 0.8 else None
    b = test_norm.rows_of(seed + 3, 1, width, wt)[0] if rng.random() < 0.8 else None
    dx, ddy = placed(rng, x.cuda()), placed(rng, dy.cuda())
    out = tg.layer_norm(dx, w.cuda() if w is not None else None, b.cuda() if b is not None else None, stats=True)
    test_norm.check_forward(x, w, b, out)
    mean, rstd = out[1], out[2]
    got = tg.layer_norm_backward(ddy, dx, mean, rstd, w.cuda() if w is not None else None)
    args = (dy, x, mean.cpu(), rstd.cpu(), w)
    for name, g, r, bound in zip(("dx", "dweight", "dbias"), got, ref.layer_norm_backward(*args),
                                 ref.layer_norm_backward_bounds(*args)):
        test_norm.within(g, r, bound, name)


def ffn_case(tg, rng):
    while True:
        tokens, width, hidden = log_int(rng, 1, 6000), 8 * log_int(rng, 1, 600), 8 * log_int(rng, 1, 1200)
        if tokens * width * hidden < 3e10:
            break
    act, dtype = rng.choice(test_ffn.ACTS), rng.choice(["bf16", "f16"])
    d = test_ffn.make(rng.randrange(1 << 30), tokens, width, hidden, dtype)
    for k in d:
        if rng.random() < 0.3:
            d[k] = test_ffn.widened(d[k], 8 * rng.randint(1, 4))
    _, saved = test_ffn.check_forward(tg, d, act)
    test_ffn.check_backward(tg, d, saved, act)


def dropout_case(tg, rng):
    n, skip = log_int(rng, 1, 20000), rng.choice([0, 0, 1, 3, 8])
    dt = ref.DTYPES[rng.choice(["bf16", "f16", "f32"])]
    p, seed, offset = rng.choice([0.0, 0.1, 0.5, rng.random()]), rng.getrandbits(64), rng.getrandbits(64)
    x, res = torch.randn(n + skip).to(dt), torch.randn(n + skip).to(dt) if rng.random() < 0.5 else None
    y = tg.dropout(x.cuda()[skip:], p, seed, offset, residual=res.cuda()[skip:] if res is not None else None)
    from tests import test_dropout

    test_dropout.check(y, x[skip:], res[skip:] if res is not None else None, p, seed, offset)


def test_random_operators(cuda_lib):
    rng = random.Random(SEED)
    for i in range(CASES):
        kind = rng.choice([norm_case, ffn_case, ffn_case, dropout_case])
        state = rng.getstate()
        try:
            kind(cuda_lib, rng)
        except AssertionError as e:
            raise AssertionError(f"case {i} of seed {SEED} ({kind.__name__}, generator state hash {hash(state)}): {e}") from e
