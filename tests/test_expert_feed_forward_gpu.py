"""The example block: its gradients against differences of its definition in 64 bits,
training that lowers the loss, and one token giving what it gives in a batch."""
import os
import sys

import pytest
import torch

import precision_gemm_gb300 as pg
from tests import _layers_ref as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_feed_forward as ff  # noqa: E402

pytestmark = pytest.mark.gpu


def _block64(x, params, balance, ids):
    """The block in 64 bits with the choice of experts held."""
    weights = torch.gather(torch.sigmoid(x @ params["router"].t()), 1, ids)
    weights = weights / weights.sum(1, keepdim=True)
    y = x.clone()
    for j in range(ids.shape[1]):
        for e in range(params["w1"].shape[0]):
            m = ids[:, j] == e
            h = R.act(x[m] @ params["w1"][e].t() + params["b1"][e], "gelu")
            y[m] += weights[m, j, None] * (h @ params["w2"][e].t() + params["b2"][e])
    return y


def test_block_gradients_against_differences():
    """Directional differences in 64 bits, step 1e-5: their error is of order 1e-9 of the
    loss, that of the chained FP32 gradients 1e-5 of the terms' sizes."""
    tokens, width = 50, 24
    block = ff.ExpertFeedForward(width, 40, 6, 2, torch.float32, seed=3)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(tokens, width, generator=g)
    y, saved = block.forward(x.cuda())
    ids = saved[3].cpu().long()
    at = {k: v.double().cpu() for k, v in block.params.items()}
    want = _block64(x.double(), at, None, ids)
    assert float((y.double().cpu() - want).norm() / want.norm()) < 1e-5
    dy = torch.randn(tokens, width, generator=g)
    dx, grads = block.backward(dy.cuda(), saved)

    def loss(x, params):
        return float((_block64(x, params, None, ids) * dy.double()).sum())

    h = 1e-5
    for name, grad in [("x", dx), *grads.items()]:
        u = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        sides = []
        for s in (h, -h):
            moved = dict(at)
            if name != "x":
                moved[name] = at[name] + s * u
            sides.append(loss(x.double() + (s * u if name == "x" else 0.0), moved))
        diff = (sides[0] - sides[1]) / (2 * h)
        grad = grad.double().cpu()
        assert abs(diff - float((grad * u).sum())) <= 5e-5 * float((grad.abs() * u.abs()).sum()), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_learns_and_decodes(dtype):
    teacher = ff.ExpertFeedForward(128, 256, 8, 2, dtype, seed=7)
    block = ff.ExpertFeedForward(128, 256, 8, 2, dtype, seed=8)
    losses, counts = ff.train(block, teacher, 512, 128, 25)
    assert losses[-1] < 0.9 * losses[0]
    assert int(counts.sum()) == 1024
    x = torch.randn(64, 128, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    batch, _ = block.forward(x)
    # a token alone runs on other kernels than in the batch: equal to a few roundings of its values
    tol = 2.0 ** -6 if dtype == torch.bfloat16 else 2.0 ** -16
    for t in (0, 17, 63):
        alone, _ = block.forward(x[t:t + 1].contiguous())
        assert float((alone.float() - batch[t:t + 1].float()).norm() / batch[t].float().norm()) < tol
    assert pg.device_status() == 0
