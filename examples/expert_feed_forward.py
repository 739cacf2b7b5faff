"""A feed-forward block of routed experts, trained and then decoded from, on the
library's layer calls: linear -> route -> expert_plan -> expert_linear (up, gelu) ->
expert_linear (down) -> expert_combine, and the same chain backwards.

    python examples/expert_feed_forward.py [--dtype bfloat16] [--tokens 2048] [--steps 30]

The block learns to reproduce a random teacher block of the same shape.  Every step
prints nothing; the losses at the start and the end, the largest share of an expert
and the time per step are printed at the end.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import precision_gemm_gb300 as pg  # noqa: E402


class ExpertFeedForward:
    """y = x + sum over the token's experts of weight * (w2[e] gelu(w1[e] x + b1[e]) + b2[e])."""

    def __init__(self, width, hidden, experts, top, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).to(dtype)

        self.experts, self.top = experts, top
        self.params = {"router": normal(experts, width, std=width ** -0.5),
                       "w1": normal(experts, hidden, width, std=width ** -0.5),
                       "b1": torch.zeros(experts, hidden, dtype=dtype, device=device),
                       "w2": normal(experts, width, hidden, std=hidden ** -0.5),
                       "b2": torch.zeros(experts, width, dtype=dtype, device=device)}
        self.balance = torch.zeros(experts, device=device)  # steers the choice of experts, not their weights

    def forward(self, x):
        """y for x (tokens, width), and what backward needs."""
        p = self.params
        logits = pg.linear(x, p["router"])
        weights, ids = pg.route(logits, self.top, "sigmoid", bias=self.balance)
        plan = pg.expert_plan(ids, self.experts)
        h, z = pg.expert_linear(x, p["w1"], plan, p["b1"], "gelu", gather=True, preact=True)
        o = pg.expert_linear(h, p["w2"], plan, p["b2"])
        y = pg.expert_combine(o, plan, weights, residual=x)
        return y, (x, logits, weights, ids, plan, h, z, o)

    def backward(self, dy, saved):
        """(dx, gradients of the parameters) for dy (tokens, width)."""
        p = self.params
        x, logits, weights, ids, plan, h, z, o = saved
        do, dweights = pg.expert_combine_backward(dy, o, plan, weights)
        dh, dw2, db2 = pg.expert_linear_backward(do, h, p["w2"], plan)
        dx_experts, dw1, db1 = pg.expert_linear_backward(dh, x, p["w1"], plan, "gelu", z, gather=True)
        dlogits = pg.route_backward(dweights, logits, ids, "sigmoid")
        dx_router, drouter, _ = pg.linear_backward(dlogits, x, p["router"], bias=False)
        return dy + dx_experts + dx_router, {"router": drouter, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}

    def rebalance(self, counts, rate):
        """Experts with more than their share become a little less likely to be chosen."""
        counts = counts.float()
        self.balance += rate * torch.sign(counts.mean() - counts)


def train(block, teacher, tokens, width, steps, lr=0.05, seed=1):
    """Losses of `steps` steps of momentum descent towards the teacher's outputs."""
    dtype = block.params["w1"].dtype
    g = torch.Generator(device="cuda").manual_seed(seed)
    master = {k: v.float() for k, v in block.params.items()}  # FP32 copies take the updates
    speed = {k: torch.zeros_like(v) for k, v in master.items()}
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").to(dtype)
        target, _ = teacher.forward(x)
        y, saved = block.forward(x)
        error = y.float() - target.float()
        losses.append(error.square().mean())
        _, grads = block.backward((error * (2.0 / tokens)).to(dtype), saved)
        for k, v in grads.items():
            speed[k].mul_(0.9).add_(v.float())
            master[k].sub_(lr * speed[k])
            block.params[k] = master[k].to(dtype)
        block.rebalance(saved[4].counts, 1e-3)
    return torch.stack(losses).tolist(), saved[4].counts


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", choices=("bfloat16", "float32"), default="bfloat16")
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=2)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    dtype = getattr(torch, a.dtype)
    teacher = ExpertFeedForward(a.width, a.hidden, a.experts, a.top, dtype, seed=7)
    block = ExpertFeedForward(a.width, a.hidden, a.experts, a.top, dtype, seed=8)
    train(block, teacher, a.tokens, a.width, 2)  # loads kernels, sizes the workspace
    torch.cuda.synchronize()
    t = time.perf_counter()
    losses, counts = train(block, teacher, a.tokens, a.width, a.steps)
    torch.cuda.synchronize()
    step = (time.perf_counter() - t) / a.steps
    one = torch.randn(1, a.width, device="cuda").to(dtype)
    y, _ = block.forward(one)  # a decoding step: the same calls on one token
    assert torch.isfinite(y).all() and pg.device_status() == 0
    print("loss %.4f -> %.4f in %d steps, largest expert %.2f of the mean, %.3f ms per step"
          % (losses[0], losses[-1], a.steps, float(counts.max()) / float(counts.float().mean()), 1e3 * step))


if __name__ == "__main__":
    main()
