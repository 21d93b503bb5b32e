"""Plans of the gated feed-forward block: what a caller learns of a failure,
calls under graph capture, and argument types."""

import pytest
import torch

import software_pipelined_tiled_02_gb300 as tg_host
from tests import test_ffn


def call(tg, d, **kw):
    return tg.gated_ffn(d["x"], d["wg"], d["wu"], d["wd"], **kw)


@pytest.mark.gpu
def test_a_failure_under_gated_ffn_can_be_seen(cuda_lib):
    """gated_ffn() keeps its plans to itself; gated_ffn_status() reads and clears their status words."""
    from software_pipelined_tiled_02_gb300 import operators

    tg, d = cuda_lib, test_ffn.make(3, 300, 232, 440, "bf16")
    want = call(tg, d)
    torch.cuda.synchronize()
    assert tg.gated_ffn_status()[0] == tg.OK
    plan = operators._ffn_plans[232, 440, torch.bfloat16, "silu", 0]
    plan.set_watchdog_ns(20_000_000)
    plan.debug_stall(True)
    call(tg, d)
    torch.cuda.synchronize()
    plan.debug_stall(False)
    plan.set_watchdog_ns(0)
    code, detail = tg.gated_ffn_status()
    assert code == tg.ERR_TIMEOUT and detail[0] == tg.ERR_TIMEOUT
    assert tg.gated_ffn_status()[0] == tg.OK  # cleared
    assert torch.equal(call(tg, d), want)
    torch.cuda.synchronize()
    assert tg.gated_ffn_status()[0] == tg.OK


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,width,hidden", [(3, 88, 104), (40, 120, 1000), (600, 168, 312)])
def test_first_call_of_a_size_inside_a_capture(cuda_lib, tokens, width, hidden):
    """The plan that the call makes, and one that is closed meanwhile, leave the capture whole."""
    tg, d = cuda_lib, test_ffn.make(5, tokens, width, hidden, "f16")
    torch.cuda.synchronize()
    other = tg.GatedFFN(width, hidden, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, saved = call(tg, d, save=True)
        got = (y, *saved, *tg.gated_ffn_backward(d["dy"], d["x"], d["wg"], d["wu"], d["wd"], saved))
        other.close()
    graph.replay()
    torch.cuda.synchronize()
    y, saved = call(tg, d, save=True)
    want = (y, *saved, *tg.gated_ffn_backward(d["dy"], d["x"], d["wg"], d["wu"], d["wd"], saved))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_wrong_types_of_tensors(cuda_lib):
    d = test_ffn.make(7, 10, 64, 72, "bf16")
    for dt in (torch.float64, torch.int32, torch.complex64):
        with pytest.raises(TypeError):
            cuda_lib.gated_ffn(d["x"].to(dt), d["wg"], d["wu"], d["wd"])


def test_wrong_types_of_a_plan():
    for dt in ("f64", torch.float64, None):
        with pytest.raises(TypeError):
            tg_host.GatedFFN(64, 72, dt)
    for sizes in ((64.5, 72), (64, "72")):
        with pytest.raises(TypeError):
            tg_host.GatedFFN(*sizes)
