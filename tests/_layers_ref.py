"""The layer operators' definitions in 64 bits, for the tests: plain loops over
experts and elementary functions, nothing shared with the library."""
import math

import torch

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.where(torch.isnan(z), z, torch.zeros_like(z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def dact(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p + z * p * (1 - p)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        u = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def linear(x, w, bias, name, residual):
    """(y, z, den): the layer, its pre-activation, and sum|x w| + |bias|."""
    x, w = x.double(), w.double()
    z, den = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, den = z + bias.double(), den + bias.double().abs()
    y = act(z, name)
    return (y if residual is None else y + residual.double()), z, den


def linear_backward(dy, x, w, name, z):
    """dx, dw, dbias and the sums of their terms' magnitudes.  An activation's derivative
    is formed in FP32 from values near 1, to within 2^-20 whatever its size: an eighth
    added to its magnitude makes the bound of 1e-5 cover that."""
    slope = dact(z.double(), name)
    d = dy.double() * slope
    m = dy.double().abs() * (slope.abs() + (0.0 if name in ("none", "relu") else 0.125))
    x, w = x.double(), w.double()
    return (d @ w, d.t() @ x, d.sum(0)), (m @ w.abs(), m.t() @ x.abs(), m.sum(0))


def lists(ids, experts):
    """counts, offsets, rows, slots by a loop over the pairs."""
    t, top = ids.shape
    members = [[] for _ in range(experts)]
    for p, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < experts:
            members[e].append(p)
    counts = [len(m) for m in members]
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    rows = [p for m in members for p in m]
    slots = [-1] * (t * top)
    for r, p in enumerate(rows):
        slots[p] = r
    rows += [-1] * (t * top - len(rows))
    return counts, offsets, rows, torch.tensor(slots, dtype=torch.int64).view(t, top).tolist()


def scores(logits, score):
    x = torch.nan_to_num(logits.double(), nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    if score == "sigmoid":
        return torch.sigmoid(x)
    m = x.max(1, keepdim=True).values
    ex = torch.where(x == m, torch.ones_like(x), torch.exp(x - m))
    ex = torch.where(x == -math.inf, torch.zeros_like(x), ex)
    s = ex.sum(1, keepdim=True)
    return torch.where(s > 0, ex / s, torch.zeros_like(ex))


# Bounds.  A product's terms are summed in FP32 in some order and blocks: the library's
# normalised bound for FP32-class products, 1e-5 of the sum of the terms' magnitudes, is
# the per-element limit.  Rounding to bfloat16 (8 significant bits) adds half a unit in
# its last place, at most 2^-8 of the value.  An activation passes an error on with a factor of at most 1.13 (the
# largest slope of the five) and adds a few roundings of its own, 2^-21 of the value.
SLOPE, NORM, HALF = 1.13, 1e-5, 2.0 ** -8


def close(got, want, den, dtype, slope=SLOPE, inner=0.0):
    """|got - want| <= slope * (1e-5 + inner) * den + 2^-21 |want| (+ 2^-8 |want| in bfloat16);
    `inner`: the relative rounding of the products' operands."""
    got = got.double().cpu()
    want, den = want.cpu(), den.cpu()
    assert got.shape == want.shape
    err = (got - want).abs()
    exact = slope * (NORM + inner) * den + 2.0 ** -21 * want.abs()
    tol = exact + (HALF * (want.abs() + exact) if dtype == torch.bfloat16 else 0.0)
    bad = ~(err <= tol + 1e-30)
    assert not bad.any(), "%d of %d off; worst ratio %g" % (int(bad.sum()), bad.numel(),
                                                           float((err / (tol + 1e-30)).max()))
