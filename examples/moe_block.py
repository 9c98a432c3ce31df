"""A transformer's MoE block in blockwise FP8: training steps, then single
tokens as a server would run them.

    python examples/moe_block.py [--tokens 8192] [--dim 2048] [--hidden 1024] [--experts 16] [--top-k 4] [--steps 5]

The block takes the residual stream x and the output u of the block before it:

    r, h = resid_norm(x, w_pre, u, w_post, gate)   r = x + gate N(u) w_post, h = N(r) w_pre
    y    = r + experts(h)                          router, dispatch, FP8 experts, combine

and is trained to move r towards a fixed random target.  Data and weights are random.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import blockwise_scaled_fp8_bs_amd as bs  # noqa: E402


class MoEBlock(torch.nn.Module):
    def __init__(self, dim, hidden, experts, top_k, checkpoint="fp8", device="cuda"):
        super().__init__()
        ones = lambda: torch.nn.Parameter(torch.ones(dim, device=device))  # noqa: E731
        self.w_post, self.w_pre = ones(), ones()
        self.gate = torch.nn.Parameter(torch.full((1, dim), 0.5, device=device))
        groups = 4 if experts % 4 == 0 and experts >= 8 and top_k <= experts // 2 else 1
        self.moe = bs.Float8BlockwiseMoE(dim, hidden, experts, top_k, score="sigmoid", n_group=groups,
                                         topk_group=max(1, groups // 2), group_best=2, checkpoint=checkpoint,
                                         device=device)

    def forward(self, x, u):
        r, h = bs.resid_norm(x, self.w_pre, u=u, w_post=self.w_post, gate=self.gate)
        return self.moe(h, residual=r)


def train(block, x, u, target, steps, rate=0.02, balance_rate=1e-3):
    """SGD steps on mean |y - target|^2; the router's bias moves towards even loads."""
    losses = []
    for _ in range(steps):
        y = block(x, u)
        loss = (y.float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss * y.numel() / y.shape[0], list(block.parameters()))
        with torch.no_grad():
            for p, g in zip(block.parameters(), grads):
                p.sub_((rate * g.float()).to(p.dtype))
            load = block.moe.last_counts.float()
            block.moe.balance.add_(balance_rate * torch.sign(load.mean() - load))
        losses.append(loss.detach())
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 8192), ("dim", 2048), ("hidden", 1024), ("experts", 16), ("top-k", 4), ("steps", 5)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--checkpoint", choices=("fp8", "bf16"), default="fp8", help="how [a | b] is kept for the backward")
    a = ap.parse_args()
    if not torch.cuda.is_available():
        sys.exit("this example needs an MI355X")
    torch.manual_seed(0)
    block = MoEBlock(a.dim, a.hidden, a.experts, a.top_k, a.checkpoint)
    new = lambda n, s: (torch.randn(n, a.dim, device="cuda") * s).to(torch.bfloat16)  # noqa: E731
    x, u, target = new(a.tokens, 1.0), new(a.tokens, 1.0), new(a.tokens, 1.0)
    train(block, x, u, target, 1)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    t = time.perf_counter()
    losses = train(block, x, u, target, a.steps)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) / a.steps * 1e3
    print(f"training: {a.tokens} tokens, {ms:.2f} ms a step, "
          f"{torch.cuda.max_memory_allocated() / 2 ** 20:.0f} MiB at the peak, loss " + " ".join(f"{v:.4f}" for v in losses))
    block.eval()
    block.moe.prepare_serving()
    with torch.no_grad():
        for n in (1, 32):
            xs, us = new(n, 1.0), new(n, 1.0)
            graph = torch.cuda.CUDAGraph()
            block(xs, us)
            with torch.cuda.graph(graph):
                y = block(xs, us)
            took = []
            for step in (lambda: block(xs, us), graph.replay):
                step()
                torch.cuda.synchronize()
                t = time.perf_counter()
                for _ in range(100):
                    step()
                torch.cuda.synchronize()
                took.append((time.perf_counter() - t) * 1e4)
            print(f"serving: {n} token(s), {took[0]:.0f} us a pass, {took[1]:.0f} us replayed from a graph, "
                  f"|y| {float(y.float().norm()):.3f}")


if __name__ == "__main__":
    main()
