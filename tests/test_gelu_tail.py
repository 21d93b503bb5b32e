"""gelu far below zero, where the activation is the product of a gate and a
tiny probability: every kernel of the block against 64 bits, relatively.

The activation is formed from Q(g) = exp(-g^2/2) R(|g|), the normal
distribution's tail.  R carries at most 1e-5 relatively (its approximation, the
reciprocal in it, and fp32 steps); the exponent -g^2/2 is rounded three times,
each by 2^-24 relatively, so the exponential is off by 3 (g^2/2) 2^-24 < 1e-7 g^2
and by 2^-22 of its own.  2e-7 g^2 leaves a factor of two.  All gates, u and dh
below are exact in 16 bits, so nothing else enters but the roundings to 16 bits.
"""

import pytest
import torch

from tests import operator_reference as ref
from tests.test_ffn import U, within

pytestmark = pytest.mark.gpu

# fp16 down to where gelu(g) 2^15 leaves its normal numbers; bf16 to where exp(-g^2/2) leaves fp32's
GATES = {"f16": [-1.0, -2.0, -3.0, -3.5, -4.0, -4.5, -5.0, -5.5, -6.0],
         "bf16": [-1.0, -3.0, -4.0, -5.0, -6.0, -7.0, -8.0, -9.0, -10.0, -12.0, -13.0]}
SIZES = [(7, 64, 64), (11, 64, 64), (11, 8, 4984), (13, 1024, 64), (70, 264, 512), (300, 64, 96), (700, 256, 1024)]


def relative(g):
    return 1e-5 + 2e-7 * g * g


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,width,hidden", SIZES)
def test_far_negative_gates(cuda_lib, tokens, width, hidden, dtype):
    dt = ref.DTYPES[dtype]
    gates = torch.tensor(GATES[dtype], device="cuda")
    g1 = gates.repeat(tokens // len(gates) + 1)[:tokens]
    x = torch.zeros(tokens, width, device="cuda", dtype=dt)
    x[:, 0], x[:, 1] = g1.to(dt), 128
    wg, wu = (torch.zeros(hidden, width, device="cuda", dtype=dt) for _ in range(2))
    wg[:, 0], wu[:, 1] = 1, 256  # u = 2^15
    wd = torch.zeros(width, hidden, device="cuda", dtype=dt)
    wd[0] = 2.0 ** -6
    dy = torch.zeros_like(x)
    dy[:, 0] = 2.0 ** 6  # dh = 1
    y, saved = cuda_lib.gated_ffn(x, wg, wu, wd, "gelu", save=True)
    g = g1.double()
    assert torch.equal(saved[0].double(), g[:, None].expand(-1, hidden)) and bool((saved[1] == 2.0 ** 15).all())

    largest = 60000 if dtype == "f16" else 1e30

    def rounded(v, off):  # an error of `off` before the rounding to 16 bits
        return off + 1.01 * ref.u_out(dt) * (v.abs() + off) + ref.tiny(dt)

    a, slope = ref.activation(g, "gelu")
    h = a * 2.0 ** 15
    hb = rounded(h, relative(g) * h.abs())
    within(saved[2], h[:, None].expand(-1, hidden), hb[:, None].expand(-1, hidden), "h")
    sums = (hidden / 16 + 16) * 2 * U  # an fp32 sum over the hidden units
    one_y = hidden * h * 2.0 ** -6
    yb = hidden * 2.0 ** -6 * hb + sums * (one_y.abs() + hidden * 2.0 ** -6 * hb)
    fits = one_y.abs() + yb < largest
    within(y[fits, 0], one_y[fits], rounded(one_y, yb)[fits], "y")

    # dh = 1 in every unit: dx[:, 0] sums dg over the units, dx[:, 1] sums 256 du
    dx = cuda_lib.gated_ffn_backward(dy, x, wg, wu, wd, saved, "gelu")[0]
    spread = ref.cdf(g) + g.abs() * torch.exp(-g * g / 2) * 0.3989422804014327  # the slope's two terms, which have opposite signs
    dg, du = slope * 2.0 ** 15, a
    for column, one, off, weight in ((0, dg, relative(g) * spread * 2.0 ** 15, 1.0), (1, du, relative(g) * a.abs(), 256.0)):
        total = hidden * weight * one
        each = hidden * weight * rounded(one, off)
        fits = total.abs() + each < largest
        bound = rounded(total, each + sums * (total.abs() + each))
        within(dx[fits, column], total[fits], bound[fits], f"dx column {column}")
