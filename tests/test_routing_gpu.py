"""Routing to experts against its definition in 64 bits: ties, groups, the balance
bias, masked tokens, rows of -infinity and NaN, and the gradient of the logits."""
import math

import pytest
import torch

import precision_gemm_gb300 as pg
from tests import _layers_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
IDS = {torch.float32: "f32", torch.bfloat16: "bf16"}
# Weights: an exponential or two, a division, a sum of at most 32 terms and another
# division, each good to 2 units of 2^-24: 2^-19 covers them all.
WEIGHT = 2.0 ** -19


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _choose(choice, top, groups, group_top):
    """Indices of the best choices by stable sorting, groups first."""
    t, e = choice.shape
    if groups > 1:
        per = choice.view(t, groups, -1)
        best = per.topk(min(2, e // groups), 2).values.sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :group_top]
        inside = torch.zeros(t, groups, dtype=torch.bool).scatter_(1, keep, True)
        choice = torch.where(inside.repeat_interleave(e // groups, 1), choice, -math.inf)
    return torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :top]


def _weights(p, ids, renorm, scale):
    w = torch.gather(p, 1, ids)
    if renorm:
        s = w.sum(1, keepdim=True)
        w = torch.where(s > 0, w / s, torch.zeros_like(w))
    return w * scale


def _spread_logits(g, t, e, dtype):
    """Every row a permutation of values 1/16 apart, exact in both types: no near ties."""
    base = (torch.arange(e) - e // 2) / 16.0
    return torch.stack([base[torch.randperm(e, generator=g)] for _ in range(t)]).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,top,renorm,scale", [(1, 1, 1, True, 1.0), (3, 2, 2, False, 1.0), (8, 64, 6, True, 2.5),
                                                  (9, 33, 5, False, 0.5), (50, 100, 32, True, 1.0),
                                                  (130, 160, 8, True, 1.0), (65, 257, 3, False, 1.0),
                                                  (40, 512, 32, True, 1.0)])
def test_route(dtype, score, t, e, top, renorm, scale):
    if score == "sigmoid" and e > 256:
        e, top = 256, min(top, 16)  # beyond, sigmoids of the grid's largest logits meet in 32 bits
    logits = _spread_logits(_gen(t + e), t, e, dtype)
    weights, ids = pg.route(logits.cuda(), top, score, renormalize=renorm, scale=scale)
    want = _choose(logits.double(), top, 1, 1)
    assert torch.equal(ids.cpu().long(), want) and ids.dtype == torch.int32
    w = _weights(R.scores(logits, score), want, renorm, scale)
    assert ((weights.double().cpu() - w).abs() <= WEIGHT * w).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,top,groups,group_top", [(20, 64, 4, 8, 2), (33, 256, 8, 8, 4), (17, 60, 6, 4, 3),
                                                      (11, 32, 3, 32, 5), (7, 96, 30, 3, 1)])
def test_route_groups_and_balance(score, t, e, top, groups, group_top):
    g = _gen(e + top)
    logits = torch.randn(t, e, generator=g)
    balance = torch.randn(e, generator=g) * 0.1
    p = R.scores(logits, score)
    choice = p + balance.double()
    want = _choose(choice, top, groups, group_top)
    # no near tie that 32-bit scores could turn, where it would change the choice: among the groups'
    # sums, and among the best choices of the groups that stay (one more than are taken)
    per = choice.view(t, groups, -1).topk(min(2, e // groups), 2).values.sum(2)
    more = torch.gather(choice, 1, _choose(choice, min(top + 1, group_top * (e // groups)), groups, group_top))
    for v in (torch.sort(per, dim=1, descending=True).values, more):
        assert v.shape[1] < 2 or float((v[:, :-1] - v[:, 1:]).min()) > 4e-7
    mask = torch.rand(t, generator=g) < 0.7
    weights, ids = pg.route(logits.cuda(), top, score, bias=balance.cuda(), groups=groups, group_top=group_top,
                            mask=mask.cuda())
    assert torch.equal(ids.cpu().long(), torch.where(mask[:, None], want, -1))
    w = torch.where(mask[:, None], _weights(p, want, True, 1.0), 0.0)
    assert ((weights.double().cpu() - w).abs() <= WEIGHT * w).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lower_index(dtype, score):
    g = _gen(9)
    logits = torch.randint(-2, 3, (64, 90), generator=g).to(dtype)  # five values: ties everywhere
    weights, ids = pg.route(logits.cuda(), 12, score)
    assert torch.equal(ids.cpu().long(), _choose(logits.double(), 12, 1, 1))
    same = torch.zeros(5, 64, dtype=dtype)
    weights, ids = pg.route(same.cuda(), 4, score, groups=8, group_top=3)
    assert ids.tolist() == [[0, 1, 2, 3]] * 5
    assert (weights == 0.25).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_rows_that_leave_nothing(score):
    e, top = 40, 4
    low = torch.finfo(torch.float32).min
    logits = torch.zeros(6, e)
    logits[0] = -math.inf                 # nothing at all
    logits[1] = -math.inf
    logits[1, 7] = 0.5                    # one expert left
    logits[2] = low                       # the type's lowest value everywhere
    logits[3] = math.nan
    logits[3, 5], logits[3, 3] = 1.0, 2.0  # NaN counts as -infinity
    logits[4, 30] = math.inf
    logits[5, :20] = low                  # half masked by the lowest value
    weights, ids = pg.route(logits.cuda(), top, score)
    weights, ids = weights.cpu(), ids.cpu()
    assert (ids >= 0).all() and (ids < e).all()
    assert all(len(set(r)) == top for r in ids.tolist())
    assert torch.isfinite(weights).all()
    assert not weights[0].any()
    assert ids[1, 0] == 7 and weights[1].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert ids[3, :2].tolist() == [3, 5] and weights[3, 2:].tolist() == [0.0, 0.0]
    assert ids[4, 0] == 30 and ids[5].tolist() == [20, 21, 22, 23]
    if score == "softmax":
        assert ids[2].tolist() == [0, 1, 2, 3] and (weights[2] == 0.25).all()
        assert weights[4].tolist() == [1.0, 0.0, 0.0, 0.0]
    else:
        assert not weights[2].any()  # sigmoids of zero
    grads = pg.route_backward(torch.ones(6, top, device="cuda"), logits.cuda(), ids.cuda(), score)
    assert torch.isfinite(grads).all()


def _backward64(dw, logits, ids, score, renorm, scale):
    x = logits.double().requires_grad_(True)
    p = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    held = (ids >= 0) & (ids < logits.shape[1])
    q = torch.gather(p, 1, torch.where(held, ids, 0)) * held
    if renorm:
        s = q.sum(1, keepdim=True)
        q = q / torch.where(s > 0, s, torch.ones_like(s))
    return torch.autograd.grad((q * dw.double()).sum() * scale, x)[0]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,top,renorm,scale", [(1, 2, 2, False, 1.0), (5, 64, 6, True, 2.5), (9, 33, 5, False, 0.5),
                                                  (31, 160, 8, True, 1.0), (6, 512, 32, True, 1.0), (70, 8, 1, False, 1.0)])
def test_route_backward(dtype, score, t, e, top, renorm, scale):
    g = _gen(t * e)
    logits = (torch.randn(t, e, generator=g) * 2).to(dtype)
    ids = _choose(logits.double(), top, 1, 1)
    if t > 5:
        ids[2] = -1          # a masked token
        ids[3, 0] = e + 5    # no expert
    dw = torch.randn(t, top, generator=g)
    got = pg.route_backward(dw.cuda(), logits.cuda(), ids.to(torch.int32).cuda(), score, renormalize=renorm, scale=scale)
    want = _backward64(dw, logits, ids, score, renorm, scale)
    assert got.dtype == dtype
    # terms cancel: each is at most the largest |dw| scale / sum(q) times p, good to 2^-18
    p = R.scores(logits, score)
    held = (ids >= 0) & (ids < e)
    total = (torch.gather(p, 1, torch.where(held, ids, 0)) * held).sum(1, keepdim=True)
    size = p * dw.double().abs().sum(1, keepdim=True) * scale * (2 / total.clamp_min(1e-30) if renorm else 2)
    tol = 2.0 ** -18 * size + (R.HALF * want.abs() if dtype == torch.bfloat16 else 0.0)
    off = (got.double().cpu() - want).abs()
    assert (off <= tol + 1e-30).all(), float((off / (tol + 1e-30)).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_against_differences(score):
    """Directional differences of the weights in 64 bits with the choice held; step 1e-5."""
    t, e, top, h = 12, 24, 4, 1e-5
    g = _gen(1)
    logits = torch.randn(t, e, generator=g)
    dw = torch.randn(t, top, generator=g)
    _, ids = pg.route(logits.cuda(), top, score)
    grad = pg.route_backward(dw.cuda(), logits.cuda(), ids, score).double().cpu()
    u = torch.randn(t, e, generator=g, dtype=torch.float64)

    def loss(x):
        return float((_weights(R.scores(x, score), ids.cpu().long(), True, 1.0) * dw.double()).sum())

    diff = (loss(logits.double() + h * u) - loss(logits.double() - h * u)) / (2 * h)
    assert abs(diff - float((grad * u).sum())) <= 1e-5 * float((grad.abs() * u.abs()).sum())


def test_route_strided_logits_and_no_tokens():
    wide = torch.full((10, 70), math.nan, device="cuda")
    wide[:, 3:67] = torch.randn(10, 64, generator=_gen(3)).cuda()
    view = wide[:, 3:67]
    w, i = pg.route(view, 5)
    w2, i2 = pg.route(view.contiguous(), 5)
    assert torch.equal(w, w2) and torch.equal(i, i2)
    w, i = pg.route(torch.empty(0, 64, device="cuda"), 5)
    assert w.shape == i.shape == (0, 5)
    assert pg.route_backward(torch.empty(0, 5, device="cuda"), torch.empty(0, 64, device="cuda"), i).shape == (0, 64)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("low", [-60.0, -80.0, -86.0])
def test_route_backward_of_renormalised_weights_of_tiny_scores(score, low):
    """Chosen experts (by the balance bias) whose scores are close to the smallest floats: their
    renormalised weights, and so the gradients, are of the usual size.  Each is a score's ratio:
    the scores' relative errors (2^-21, and 2^-23 / 2^-126 of a half unit near the smallest normal
    float) times the sizes of dw, and the rounding of the ratios' sums."""
    t, e, top = 9, 64, 6
    g = _gen(int(-low))
    logits = low - torch.rand(t, e, generator=g)
    if score == "softmax":
        logits[:, e - 1] = 0.0  # takes all of the softmax
    dw = torch.randn(t, top, generator=g) * 100
    balance = torch.zeros(e)
    balance[:top] = 4.0
    weights, ids = pg.route(logits.cuda(), top, score, bias=balance.cuda(), scale=2.5)
    assert int(ids.max()) < top
    x = logits.double()
    q = torch.gather(torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x), 1, ids.cpu().long())
    w = q / q.sum(1, keepdim=True)
    assert ((weights.cpu().double() - 2.5 * w).abs() <= 2.0 ** -18 * 2.5 * w).all()
    got = pg.route_backward(dw.cuda(), logits.cuda(), ids, score, scale=2.5)
    d = 2.5 * w * (dw.double() - (w * dw.double()).sum(1, keepdim=True)) * (1 - q if score == "sigmoid" else 1)
    want = torch.zeros(t, e, dtype=torch.float64).scatter_(1, ids.cpu().long(), d)
    assert ((got.double().cpu() - want).abs() <= 2.0 ** -17 * 2.5 * dw.double().abs().sum(1, keepdim=True)).all()


def test_counts_are_checked_before_results_are_allocated():
    logits, ids = torch.zeros(1, 16, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    for call in (lambda: pg.route(logits, 1 << 24), lambda: pg.expert_plan(ids, 1 << 24)):
        with pytest.raises(pg.SgemmError):
            call()
    for call in (lambda: pg.route(logits, (1 << 32) + 2), lambda: pg.expert_plan(ids, (1 << 32) + 2),
                 lambda: pg.route(logits, 2, groups=(1 << 32) + 1),
                 lambda: pg.route(logits, 2, groups=2, group_top=(1 << 32) + 1)):
        with pytest.raises(ValueError):  # beyond the 32 bits of the library's argument
            call()
    assert torch.cuda.max_memory_allocated() - held < 1 << 20
