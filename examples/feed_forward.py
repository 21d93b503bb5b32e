"""A transformer's pre-norm feed-forward sub-block on the library's operators:

    out = x + dropout(ffn(layer_norm(x)))

trained on synthetic data through torch's autograd, then served one token at a
time.  Run it on a GB300:

    python examples/feed_forward.py [--tokens 4096] [--width 1024] [--hidden 4096] [--steps 30]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import software_pipelined_tiled_02_gb300 as tg  # noqa: E402


class FeedForward(torch.autograd.Function):
    """The sub-block as one autograd node: the operators' own backward passes, and the dropout mask formed again
    from (seed, offset)."""

    @staticmethod
    def forward(ctx, x, norm_w, norm_b, w_gate, w_up, w_down, activation, p, seed, offset):
        n, mean, rstd = tg.layer_norm(x, norm_w, norm_b, stats=True)
        y, saved = tg.gated_ffn(n, w_gate, w_up, w_down, activation, save=True)
        ctx.save_for_backward(x, norm_w, w_gate, w_up, w_down, n, mean, rstd, *saved)
        ctx.rest = (activation, p, seed, offset)
        return tg.dropout(y, p, seed, offset, residual=x)

    @staticmethod
    def backward(ctx, dout):
        x, norm_w, w_gate, w_up, w_down, n, mean, rstd, *saved = ctx.saved_tensors
        activation, p, seed, offset = ctx.rest
        dout = dout.contiguous()
        dy = tg.dropout_backward(dout, p, seed, offset)
        dn, dw_gate, dw_up, dw_down = tg.gated_ffn_backward(dy, n, w_gate, w_up, w_down, tuple(saved), activation)
        dx, dnorm_w, dnorm_b = tg.layer_norm_backward(dn, x, mean, rstd, norm_w)
        return dx + dout, dnorm_w, dnorm_b, dw_gate, dw_up, dw_down, None, None, None, None


class Block(torch.nn.Module):
    def __init__(self, width, hidden, activation="silu", p=0.1, seed=0, dtype=torch.bfloat16):
        super().__init__()
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return torch.nn.Parameter((torch.randn(rows, cols, generator=gen, device="cuda") * cols ** -0.5).to(dtype))

        self.norm_w = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.norm_b = torch.nn.Parameter(torch.zeros(width, device="cuda"))
        self.w_gate, self.w_up, self.w_down = weight(hidden, width), weight(hidden, width), weight(width, hidden)
        self.activation, self.p, self.seed, self.calls = activation, p, seed, 0

    def forward(self, x):
        if not self.training:  # no mask, nothing saved; a few tokens take the weight-streaming kernels
            n = tg.layer_norm(x, self.norm_w, self.norm_b)
            return x + tg.gated_ffn(n, self.w_gate, self.w_up, self.w_down, self.activation)
        self.calls += 1  # every step draws another mask
        return FeedForward.apply(x, self.norm_w, self.norm_b, self.w_gate, self.w_up, self.w_down, self.activation,
                                 self.p, self.seed, self.calls)


def train(block, teacher, tokens, steps, lr=2e-3, seed=1):
    """Fit the block to the teacher's outputs; the losses of all steps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    master = {name: w.detach().float() for name, w in block.named_parameters()}  # updates are smaller than bf16's steps
    moments = {name: (torch.zeros_like(m), torch.zeros_like(m)) for name, m in master.items()}
    width, dtype = block.w_gate.shape[1], block.w_gate.dtype
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
        with torch.no_grad():
            want = teacher(x).float()
        loss = (block(x).float() - want).square().mean()
        block.zero_grad(set_to_none=True)
        loss.backward()
        losses.append(loss.detach())
        with torch.no_grad():  # Adam on the fp32 copies
            for name, w in block.named_parameters():
                a, b = moments[name]
                g = w.grad.float()
                a.mul_(0.9).add_(g, alpha=0.1)
                b.mul_(0.99).addcmul_(g, g, value=0.01)
                rate = lr * (1 - 0.99 ** step) ** 0.5 / (1 - 0.9 ** step)
                master[name].addcdiv_(a, b.sqrt().add_(1e-8), value=-rate)
                w.copy_(master[name])
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    teacher = Block(a.width, a.hidden, seed=7).eval()
    block = Block(a.width, a.hidden, p=0.05)
    losses = train(block, teacher, a.tokens, a.steps)
    print("loss: first %.4f, last %.4f" % (losses[0], losses[-1]))
    block.eval()
    x = torch.randn(8, a.width, device="cuda").to(block.w_gate.dtype)
    together, single = block(x), torch.cat([block(x[i:i + 1]) for i in range(len(x))])
    print("8 tokens together and one at a time: largest difference %.3g" % float((together - single).abs().max()))


if __name__ == "__main__":
    main()
