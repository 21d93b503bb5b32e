"""The operators together, as examples/feed_forward.py runs them."""

import importlib.util
import os

import pytest
import torch

from tests import operator_reference as ref
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_lowers_the_loss(cuda_lib, example):
    teacher = example.Block(256, 512, seed=7).eval()
    block = example.Block(256, 512, p=0.0)
    losses = example.train(block, teacher, 2048, 25)
    assert losses[-1] < 0.7 * losses[0] and all(v == v for v in losses)


def test_gradients_of_the_whole_block(cuda_lib, example):
    """Against torch's autograd in 64 bits on the same values and mask.  A gradient passes at most a dozen roundings to
    bf16 on its way, each 2^-8 at most and independent, so 12 x 2^-8 bounds its relative error in norm."""
    tokens, width, hidden, p = 300, 128, 264, 0.25
    block = example.Block(width, hidden, activation="gelu", p=p, seed=5)
    with torch.no_grad():
        block.norm_w.add_(0.1 * torch.randn(width, device="cuda"))
        block.norm_b.add_(0.1 * torch.randn(width, device="cuda"))
    x = torch.randn(tokens, width, device="cuda").bfloat16().requires_grad_()
    dout = torch.randn(tokens, width, device="cuda").bfloat16()
    block(x).backward(dout)
    kept = torch.from_numpy(ref.dropout_kept(0, tokens * width, p, 5, 1)).view(tokens, width).cuda()
    names = ["norm_w", "norm_b", "w_gate", "w_up", "w_down"]
    v = {k: getattr(block, k).detach().double().requires_grad_() for k in names}
    xd = x.detach().double().requires_grad_()
    n = torch.nn.functional.layer_norm(xd, (width,), v["norm_w"], v["norm_b"])
    h = torch.nn.functional.gelu(n @ v["w_gate"].T) * (n @ v["w_up"].T)
    (xd + (h @ v["w_down"].T) * kept / (1 - p)).backward(dout.double())
    for name, got, want in [("x", x.grad, xd.grad)] + [(k, getattr(block, k).grad, v[k].grad) for k in names]:
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 12 * 2.0 ** -8, (name, off)


def test_serving_one_token_at_a_time(cuda_lib, example):
    """The same function whatever the number of tokens, up to the order of the sums."""
    for width, hidden in ((512, 1024), (2048, 4096)):
        block = example.Block(width, hidden, seed=3).eval()
        x = torch.randn(40, width, device="cuda").bfloat16()
        with torch.no_grad():
            together = block(x)
            single = torch.cat([block(x[i:i + 1]) for i in range(40)])
        off = (together.float() - single.float()).abs()
        # at most one rounding of h and one of y differ, by an ulp each; y stays below 8
        assert float(off.max()) <= 8 * 2.0 ** -7


def test_command_line(cuda_lib):
    import subprocess
    import sys

    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "feed_forward.py"), "--tokens", "512", "--width", "128",
                        "--hidden", "256", "--steps", "3"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "loss: first" in r.stdout
