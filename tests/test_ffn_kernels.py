"""Every kernel that a product of the gated block can take, each with its
outputs between bands that must not change, and with its pipeline stalled.

The cost model picks the kernels; `GatedFFN.kernels` says which, and each size
below names the one that it is here for, so a change of the model that loses a
kernel's coverage fails instead of passing in silence.
"""

import os
import subprocess
import sys

import pytest
import torch

from tests.conftest import ROOT
from tests.test_ffn import DT, backward_reference, forward_reference, make, within

pytestmark = pytest.mark.gpu

# (product, kernel, CTAs of a cluster): (tokens, width, hidden), none of them whole tiles
SIZES = {
    ("up", "rows", 1): (5, 72, 88), ("down", "rows", 1): (8, 136, 264),
    ("up", "few", 1): (11, 8, 4984), ("up", "few", 2): (10, 368, 8), ("up", "few", 4): (9, 520, 8),
    ("up", "few", 8): (11, 968, 8), ("up", "few", 16): (9, 2792, 8), ("up", "pairs", 2): (131, 72, 88),
    ("down", "few", 1): (26, 7392, 72), ("down", "few", 2): (9, 8, 328), ("down", "few", 4): (9, 8, 472),
    ("down", "few", 8): (9, 8, 1000), ("down", "few", 16): (11, 8, 2640), ("down", "pairs", 2): (131, 72, 88),
    ("dh", "few", 1): (1, 8, 10528), ("dh", "few", 2): (1, 328, 8), ("dh", "few", 4): (2, 456, 8),
    ("dh", "few", 8): (1, 1008, 8), ("dh", "few", 16): (1, 2656, 8), ("dh", "pairs", 2): (131, 72, 88),
    ("dx", "few", 1): (2, 1376, 8), ("dx", "few", 2): (1, 8, 72), ("dx", "few", 4): (1, 8, 200),
    ("dx", "few", 8): (1, 8, 456), ("dx", "few", 16): (1, 8, 1912), ("dx", "pairs", 2): (131, 72, 88),
    ("dw", "few", 1): (77, 6672, 16), ("dw", "few", 2): (333, 8, 8), ("dw", "few", 4): (449, 8, 8),
    ("dw", "few", 8): (962, 8, 8), ("dw", "few", 16): (3716, 8, 8), ("dw", "pairs", 2): (131, 72, 88),
}
GUARD = 4096
SENTINEL = 7.0


class Banded:
    """A [rows, cols] matrix of row distance ld inside a buffer of sentinels."""

    def __init__(self, rows, cols, dtype, pad=0):
        self.ld = cols + pad
        self.room = torch.full((GUARD + rows * self.ld + GUARD,), SENTINEL, dtype=dtype, device="cuda")
        self.view = self.room[GUARD:-GUARD].view(rows, self.ld)[:, :cols]
        self.ptr = self.view.data_ptr()

    def untouched(self):
        rest = self.room.clone()
        rest[GUARD:-GUARD].view(-1, self.ld)[:, :self.view.shape[1]] = SENTINEL
        return bool((rest == SENTINEL).all())


def test_every_kernel_has_a_size(cuda_lib):
    """Each product runs as CTA pairs and as clusters of 1 to 16 CTAs, the forward pass's also without tensor memory."""
    for (product, *kernel), (tokens, width, hidden) in SIZES.items():
        plan = cuda_lib.GatedFFN(width, hidden, "bf16")
        assert plan.kernels(tokens)[product] == tuple(kernel), (product, tokens, width, hidden, plan.kernels(tokens))
        plan.close()
    assert {k for k in SIZES} >= {(p, "few", r) for p in ("up", "down", "dh", "dx", "dw") for r in (1, 2, 4, 8, 16)}


@pytest.mark.parametrize("pad", [0, 8, 40])
@pytest.mark.parametrize("which", list(SIZES), ids=lambda k: "-".join(map(str, k)))
def test_outputs_stay_inside_their_matrices(cuda_lib, which, pad):
    """Bands around every output, and rows of y and dx that are apart."""
    tg, (tokens, D, F) = cuda_lib, SIZES[which]
    dtype, act = ("bf16", "silu") if pad != 8 else ("f16", "gelu")
    d = make(29, tokens, D, F, dtype)
    L, plan = tg.load(), tg.GatedFFN(D, F, dtype, act)
    y, dx = Banded(tokens, D, DT[dtype], pad), Banded(tokens, D, DT[dtype], pad)
    g, u, h, dg, du = (Banded(tokens, F, DT[dtype]) for _ in range(5))
    dwg, dwu, dwd = Banded(F, D, DT[dtype]), Banded(F, D, DT[dtype]), Banded(D, F, DT[dtype])
    P = {k: t.data_ptr() for k, t in d.items()}
    weights = (P["wg"], D, P["wu"], D, P["wd"], F)
    s = torch.cuda.current_stream().cuda_stream
    assert L.tgemm_ffn_forward(plan.handle, tokens, P["x"], D, *weights, y.ptr, y.ld, g.ptr, u.ptr, h.ptr, s) == tg.OK
    assert L.tgemm_ffn_backward(plan.handle, tokens, P["dy"], D, P["x"], D, *weights, g.ptr, u.ptr, h.ptr, dx.ptr, dx.ld,
                                dwg.ptr, dwu.ptr, dwd.ptr, dg.ptr, du.ptr, s) == tg.OK
    torch.cuda.synchronize()
    assert plan.status()[0] == tg.OK
    want = {**forward_reference(d, act), **backward_reference(d, (g.view, u.view, h.view), act)}
    outputs = {"y": y, "g": g, "u": u, "h": h, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}
    for name, t in outputs.items():
        within(t.view, *want[name], name)
    for name, t in {**outputs, "dg": dg, "du": du}.items():
        assert t.untouched(), name
    plan.close()


STALLED = [("up", "few", 1), ("up", "few", 4), ("down", "few", 16), ("up", "pairs", 2), ("dh", "few", 1), ("dh", "few", 8),
           ("dx", "few", 1), ("dx", "few", 16), ("dw", "few", 2), ("dw", "few", 16), ("dw", "few", 1)]


@pytest.mark.parametrize("which", STALLED, ids=lambda k: "-".join(map(str, k)))
def test_watchdog(cuda_lib, which):
    """A stalled forward and a stalled backward pass end with a status; the plan works again afterwards."""
    tg, (tokens, D, F) = cuda_lib, SIZES[which]
    d = make(31, tokens, D, F, "bf16")
    plan, w = tg.GatedFFN(D, F, "bf16", "silu"), (d["wg"], d["wu"], d["wd"])
    y, saved = plan.forward(d["x"], *w, save=True)
    want = (y, *saved, *plan.backward(d["dy"], d["x"], *w, saved))
    torch.cuda.synchronize()
    plan.set_watchdog_ns(20_000_000)
    plan.debug_stall(True)
    if any(kernel != "rows" for kernel, _ in (plan.kernels(tokens)[k] for k in ("up", "down"))):  # "rows" has no waits
        plan.forward(d["x"], *w)
        torch.cuda.synchronize()
        assert plan.status()[0] == tg.ERR_TIMEOUT
    plan.backward(d["dy"], d["x"], *w, saved)
    torch.cuda.synchronize()
    assert plan.status()[0] == tg.ERR_TIMEOUT
    plan.debug_stall(False)
    plan.set_watchdog_ns(0)
    y, saved = plan.forward(d["x"], *w, save=True)
    got = (y, *saved, *plan.backward(d["dy"], d["x"], *w, saved))
    torch.cuda.synchronize()
    assert plan.status()[0] == tg.OK and all(torch.equal(a, b) for a, b in zip(got, want))
    plan.close()


def test_debug_check_build(cuda_lib):
    """The bands against the build that checks its addresses."""
    if os.environ.get("TGEMM_LIB"):
        pytest.skip("already running against another build")
    from software_pipelined_tiled_02_gb300 import build

    env = dict(os.environ, TGEMM_LIB=build.build(debug=True))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests", "test_ffn_kernels.py"), "-q", "-x", "-m",
                        "gpu", "-k", "inside_their_matrices or every_kernel"], cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
