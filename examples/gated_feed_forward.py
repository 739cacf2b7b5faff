"""A gated feed-forward block behind a layer norm, trained and then served with 8-bit
weights, on the library's layer calls: layer_norm -> gated_linear -> linear with the
residual, the same chain backwards, and layer_norm -> quantize -> block_linear to serve.

    python examples/gated_feed_forward.py [--dtype bfloat16] [--tokens 2048] [--steps 30]

The block learns to reproduce a random teacher block of the same shape.  The losses at
the start and the end, the time per step, the served block's distance from the trained
one and the time of a single token are printed at the end.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import precision_gemm_gb300 as pg  # noqa: E402


class GatedFeedForward:
    """y = x + w2 (act(g) u) + b2, with [g u] = w1 norm(x) + b1."""

    def __init__(self, width, hidden, act="silu", dtype=torch.bfloat16, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=gen, device=device) * std).to(dtype)

        self.act = act
        self.params = {"norm": torch.ones(width, dtype=dtype, device=device),
                       "shift": torch.zeros(width, dtype=dtype, device=device),
                       "w1": normal(2 * hidden, width, std=width ** -0.5),
                       "b1": torch.zeros(2 * hidden, dtype=dtype, device=device),
                       "w2": normal(width, hidden, std=hidden ** -0.5),
                       "b2": torch.zeros(width, dtype=dtype, device=device)}

    def forward(self, x):
        """y for x (tokens, width), and what backward needs."""
        p = self.params
        h, mean, rstd = pg.layer_norm(x, p["norm"], p["shift"], stats=True)
        a, z = pg.gated_linear(h, p["w1"], p["b1"], self.act, preact=True)
        return pg.linear(a, p["w2"], p["b2"], residual=x), (x, mean, rstd, h, z, a)

    def backward(self, dy, saved):
        """(dx, gradients of the parameters) for dy (tokens, width)."""
        p = self.params
        x, mean, rstd, h, z, a = saved
        da, dw2, db2 = pg.linear_backward(dy, a, p["w2"])
        dh, dw1, db1 = pg.gated_linear_backward(da, h, p["w1"], z, self.act)
        dx, dnorm, dshift = pg.layer_norm_backward(dh, x, p["norm"], mean, rstd, residual=dy)
        return dx, {"norm": dnorm, "shift": dshift, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}


class Served:
    """The block with its matrices in 8 bits, a scale for each 128 x 128 of them."""

    def __init__(self, block):
        p = block.params
        hidden = p["w2"].shape[1]
        self.act, self.norm, self.shift, self.b2 = block.act, p["norm"], p["shift"], p["b2"]
        self.bg, self.bu = p["b1"][:hidden], p["b1"][hidden:].contiguous()
        self.gate, self.up = pg.quantize(p["w1"][:hidden], 128), pg.quantize(p["w1"][hidden:], 128)
        self.down = pg.quantize(p["w2"], 128)

    def forward(self, x):
        q, scales = pg.quantize(pg.layer_norm(x, self.norm, self.shift))
        g = pg.block_linear(q, *self.gate, self.bg, self.act, x_scales=scales, dtype=x.dtype)
        u = pg.block_linear(q, *self.up, self.bu, x_scales=scales, dtype=x.dtype)
        return pg.block_linear(g.mul_(u), *self.down, self.b2, residual=x)


def train(block, teacher, tokens, width, steps, lr=0.05, seed=1):
    """Losses of `steps` steps of momentum descent towards the teacher's outputs."""
    dtype = block.params["w1"].dtype
    gen = torch.Generator(device="cuda").manual_seed(seed)
    master = {k: v.float() for k, v in block.params.items()}  # FP32 copies take the updates
    speed = {k: torch.zeros_like(v) for k, v in master.items()}
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
        target, _ = teacher.forward(x)
        y, saved = block.forward(x)
        error = y.float() - target.float()
        losses.append(error.square().mean())
        _, grads = block.backward((error * (2.0 / tokens)).to(dtype), saved)
        for k, v in grads.items():
            speed[k].mul_(0.9).add_(v.float())
            master[k].sub_(lr * speed[k])
            block.params[k] = master[k].to(dtype)
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", choices=("bfloat16", "float32"), default="bfloat16")
    ap.add_argument("--act", choices=("silu", "gelu", "gelu_tanh", "relu"), default="silu")
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    dtype = getattr(torch, a.dtype)
    teacher = GatedFeedForward(a.width, a.hidden, a.act, dtype, seed=7)
    block = GatedFeedForward(a.width, a.hidden, a.act, dtype, seed=8)
    train(block, teacher, a.tokens, a.width, 2)  # loads kernels, sizes the workspace
    torch.cuda.synchronize()
    t = time.perf_counter()
    losses = train(block, teacher, a.tokens, a.width, a.steps)
    torch.cuda.synchronize()
    step = (time.perf_counter() - t) / a.steps
    served = Served(block)
    x = torch.randn(a.tokens, a.width, device="cuda").to(dtype)
    y, z = block.forward(x)[0].float(), served.forward(x).float()
    one = x[:1].contiguous()
    served.forward(one)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(100):
        served.forward(one)
    torch.cuda.synchronize()
    token = (time.perf_counter() - t) / 100
    assert torch.isfinite(z).all() and pg.device_status() == 0
    print("loss %.4f -> %.4f in %d steps, %.3f ms per step; served in 8 bits: %.4f of the block's own part off, "
          "%.3f ms per token" % (losses[0], losses[-1], a.steps, 1e3 * step,
                                 float((z - y).norm() / (y - x.float()).norm()), 1e3 * token))


if __name__ == "__main__":
    main()
