"""A transformer's feed-forward sub-block as a mixture of experts on the library's operators:

    out = x + sum over the chosen experts of weight * ffn_expert(layer_norm(x))

trained on synthetic data through torch's autograd, with a bias that evens out
the experts' load, then served token by token: with the 16-bit weights, and with
weights rounded to 4 bits.  Run it on a GB300:

    python examples/mixture_of_experts.py [--tokens 4096] [--width 1024] [--hidden 512] [--experts 16] [--top 2] [--steps 30]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import software_pipelined_tiled_02_gb300 as tg  # noqa: E402


class MixtureOfExperts(torch.autograd.Function):
    """The routed sub-block as one autograd node.  The choice of experts has no gradient; the router learns through the
    weights of those that were chosen."""

    @staticmethod
    def forward(ctx, x, norm_w, norm_b, router, w_gate, w_up, w_down, bias, top, activation):
        n, mean, rstd = tg.layer_norm(x, norm_w, norm_b, stats=True)
        logits = tg.gemm(n, router, out_dtype=torch.float32)
        weights, experts = tg.route(logits, top, "sigmoid", bias=bias)
        y, saved = tg.expert_ffn(n, experts, weights, w_gate, w_up, w_down, activation, save=True)
        ctx.save_for_backward(x, norm_w, router, w_gate, w_up, w_down, n, mean, rstd, logits, weights, experts, *saved)
        ctx.activation = activation
        ctx.mark_non_differentiable(experts)
        return x + y, experts

    @staticmethod
    def backward(ctx, dout, _):
        x, norm_w, router, w_gate, w_up, w_down, n, mean, rstd, logits, weights, experts, *saved = ctx.saved_tensors
        dout = dout.contiguous()
        dn, dweights, dw_gate, dw_up, dw_down = tg.expert_ffn_backward(dout, n, experts, weights, w_gate, w_up, w_down,
                                                                       tuple(saved), ctx.activation)
        dlogits = tg.route_backward(dweights, logits, experts, "sigmoid").to(n.dtype)
        drouter = dlogits.t() @ n  # few experts: small products
        dn = dn + dlogits @ router
        dx, dnorm_w, dnorm_b = tg.layer_norm_backward(dn, x, mean, rstd, norm_w)
        return dx + dout, dnorm_w, dnorm_b, drouter, dw_gate, dw_up, dw_down, None, None, None


def quantize(w, group=128):
    """4-bit weights of a stack of matrices: (packed, scales, zeros), each group's smallest and largest value at 0 and 15
    at the latest (and 0 among them)."""
    g = w.float().unflatten(-1, (-1, group))
    low, high = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
    scales = ((high - low) / 15).clamp(min=1e-8).to(w.dtype)
    zeros = (-low / scales.float()).round().clamp(0, 15)
    q = (g / scales.float()[..., None] + zeros[..., None]).round().clamp(0, 15).flatten(-2).to(torch.uint8)
    return q[..., 0::2] | q[..., 1::2] << 4, scales, zeros.to(torch.uint8)


class Block(torch.nn.Module):
    def __init__(self, width, hidden, experts, top, activation="silu", seed=0, dtype=torch.bfloat16):
        super().__init__()
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.nn.Parameter((torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(dtype))

        self.norm_w = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.norm_b = torch.nn.Parameter(torch.zeros(width, device="cuda"))
        self.router = weight(experts, width)
        self.w_gate, self.w_up = weight(experts, hidden, width), weight(experts, hidden, width)
        self.w_down = weight(experts, width, hidden)
        self.register_buffer("bias", torch.zeros(experts, device="cuda"))
        self.top, self.activation = top, activation

    def forward(self, x):
        if self.training:
            out, experts = MixtureOfExperts.apply(x, self.norm_w, self.norm_b, self.router, self.w_gate, self.w_up, self.w_down,
                                                  self.bias, self.top, self.activation)
            self.load = torch.bincount(experts.flatten(), minlength=len(self.bias))
            return out
        n = tg.layer_norm(x, self.norm_w, self.norm_b)
        weights, experts = self.route(n)
        return x + tg.expert_ffn(n, experts, weights, self.w_gate, self.w_up, self.w_down, self.activation)

    def route(self, n):
        logits = (n.float() @ self.router.float().t())  # few tokens: a product too small for a tile
        return tg.route(logits, self.top, "sigmoid", bias=self.bias)

    def balance(self, rate=0.01):
        """Experts with more than their share become less attractive, the others more."""
        load = self.load.float()
        self.bias -= rate * torch.sign(load - load.mean())

    def served(self, x, packed):
        """The block for a few tokens with 4-bit experts: `packed` holds `quantize`'s results for gate, up and down."""
        n = tg.layer_norm(x, self.norm_w, self.norm_b)
        weights, experts = self.route(n)
        gate, up = (tg.gemm_w4(n, *w, experts=experts, out_dtype=torch.float32) for w in packed[:2])
        h = (torch.nn.functional.silu(gate) * up).to(x.dtype)
        y = tg.gemm_w4(h, *packed[2], experts=experts, out_dtype=torch.float32)
        return x + (y * weights[..., None]).sum(1).to(x.dtype)


def train(block, teacher, tokens, steps, lr=2e-3, seed=1):
    """Fit the block to the teacher's outputs; the losses of all steps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    master = {name: w.detach().float() for name, w in block.named_parameters()}  # updates are smaller than bf16's steps
    moments = {name: (torch.zeros_like(m), torch.zeros_like(m)) for name, m in master.items()}
    width, dtype = block.w_gate.shape[-1], block.w_gate.dtype
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
        with torch.no_grad():
            want = teacher(x).float()
        loss = (block(x).float() - want).square().mean()
        block.zero_grad(set_to_none=True)
        loss.backward()
        block.balance()
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
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=2)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    teacher = Block(a.width, a.hidden, a.experts, a.top, seed=7).eval()
    block = Block(a.width, a.hidden, a.experts, a.top)
    losses = train(block, teacher, a.tokens, a.steps)
    print("loss: first %.4f, last %.4f" % (losses[0], losses[-1]))
    print("pairs of each expert in the last step:", block.load.tolist())
    block.eval()
    x = torch.randn(8, a.width, device="cuda").to(block.w_gate.dtype)
    with torch.no_grad():
        together, single = block(x), torch.cat([block(x[i:i + 1]) for i in range(len(x))])
        print("8 tokens together and one at a time: largest difference %.3g" % float((together - single).abs().max()))
        packed = [quantize(w) for w in (block.w_gate, block.w_up, block.w_down)]
        off = (block.served(x, packed) - together).float().norm() / (together - x).float().norm()
        print("with 4-bit experts: relative difference of the block's part %.3g" % float(off))


if __name__ == "__main__":
    main()
