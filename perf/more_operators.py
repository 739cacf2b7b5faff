"""Measured work of the operators around a feed-forward block: layer norm, the gated
up projection, and products with 8-bit weights, in the directions they are used.

A case is one pass through one operator.  `own` selects who computes it: the
operators' plain form (elementary torch operations in 32 bits, rounded once at
the end) or this package's public calls.  `exact` is the same pass from the
definitions in 64 bits.

Kinds of a case:
  norm          y = (x - mean) rstd w + b of each row, with its mean and rstd
  norm_bwd      (dx, dw, db) of norm for dy, the gradient that passes the norm by added to dx
  gated         y = act(g) u with [g u] = x w^T + b, and [g u] itself where a training step keeps it
  gated_bwd     (dx, dw, db) of gated for dy, with the saved [g u]
  block         y = act(x w^T + b) + r with w in e4m3, a scale for each 128 x 128 of it, and x
                rounded to e4m3 on the way, a scale for each 128 of a row
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"
BLOCK = 128        # values that share a scale
E4M3_MAX = 448.0


def listed():
    return [
        # Four tokens that decode together: the latency of one small launch.
        {"name": "norm decode bf16", "kind": "norm", "t": 4, "n": 4096, "dtype": "bf16", "eps": 1e-5},
        # A float32 batch through the norm before a block.
        {"name": "norm prefill f32", "kind": "norm", "t": 16384, "n": 2048, "dtype": "f32", "eps": 1e-5},
        # A training step's backward pass through the norm, with the reduction of the weight's gradient over all tokens.
        {"name": "norm backward bf16", "kind": "norm_bwd", "t": 16384, "n": 4096, "dtype": "bf16", "residual": True},
        # The repository's odd row length 777: rows start at any 4-byte boundary.
        {"name": "norm backward ragged f32", "kind": "norm_bwd", "t": 1500, "n": 777, "dtype": "f32",
         "residual": False},
        # One token through a gated up projection: a decoding step, where the weights' read time is all.
        {"name": "gated decode bf16", "kind": "gated", "t": 1, "n": 8192, "k": 4096, "dtype": "bf16", "act": "silu",
         "bias": False, "keep": False},
        # A prompt of 2048 tokens.
        {"name": "gated prefill bf16", "kind": "gated", "t": 2048, "n": 8192, "k": 4096, "dtype": "bf16",
         "act": "silu", "bias": False, "keep": False},
        # A forward step of float32 training at the repository's ragged sizes (1500 x 3000 x 777).
        {"name": "gated ragged f32", "kind": "gated", "t": 1500, "n": 1500, "k": 777, "dtype": "f32", "act": "gelu",
         "bias": True, "keep": True},
        # A training step's backward pass, 8192 tokens.
        {"name": "gated backward bf16", "kind": "gated_bwd", "t": 8192, "n": 4096, "k": 2048, "dtype": "bf16",
         "act": "silu", "bias": True},
        # The backward pass at the odd sizes 1300 x 1000 x 1500, all in float32.
        {"name": "gated backward f32", "kind": "gated_bwd", "t": 1300, "n": 1000, "k": 1500, "dtype": "f32",
         "act": "gelu", "bias": True},
        # One token through a projection whose weights are kept in 8 bits.
        {"name": "block decode", "kind": "block", "t": 1, "n": 8192, "k": 4096, "dtype": "bf16", "act": "none",
         "bias": False, "residual": True},
        # A prompt of 4096 tokens through the same projection.
        {"name": "block prefill", "kind": "block", "t": 4096, "n": 8192, "k": 4096, "dtype": "bf16", "act": "gelu",
         "bias": True, "residual": False},
        # Extents that end inside blocks of 128 and inside 16 bytes.
        {"name": "block ragged", "kind": "block", "t": 1300, "n": 1000, "k": 1500, "dtype": "bf16", "act": "silu",
         "bias": True, "residual": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _extent(rng, lo, hi):
    """A feature count: half of the draws multiples of 64, the others as they come, odd ones among them."""
    v = _log(rng, lo, hi)
    return max(lo, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    kind = rng.choice(["norm", "norm_bwd", "gated", "gated", "gated_bwd", "block", "block"])
    act = rng.choice(["none", "relu", "silu", "gelu"])
    dtype = rng.choice(["bf16", "f32"])
    if kind in ("norm", "norm_bwd"):
        n = _extent(rng, 64, 16384)
        case = {"kind": kind, "t": _log(rng, 1, min(65536, (1 << 26) // n)), "n": n, "dtype": dtype}
        if kind == "norm":
            case["eps"] = rng.choice([1e-5, 1e-6])
        else:
            case["residual"] = rng.random() < 0.5
        return case
    if kind == "gated":
        return {"kind": kind, "t": _log(rng, 1, 4096), "n": _extent(rng, 64, 4096), "k": _extent(rng, 64, 4096),
                "dtype": dtype, "act": act, "bias": rng.random() < 0.5, "keep": rng.random() < 0.5}
    if kind == "gated_bwd":
        return {"kind": kind, "t": _log(rng, 64, 8192), "n": _extent(rng, 64, 4096), "k": _extent(rng, 64, 2048),
                "dtype": dtype, "act": act, "bias": rng.random() < 0.5}
    return {"kind": kind, "t": _log(rng, 1, 8192), "n": _extent(rng, 64, 8192), "k": _extent(rng, 64, 4096),
            "dtype": "bf16", "act": act, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}


# ---- inputs ---------------------------------------------------------------------------


def _tiles(w):
    """w (n, k), padded with zeros to whole blocks, as (blocks of rows, 128, blocks of columns, 128)."""
    n, k = w.shape
    rows, cols = -(-n // BLOCK), -(-k // BLOCK)
    full = w.new_zeros(rows * BLOCK, cols * BLOCK)
    full[:n, :k] = w
    return full.view(rows, BLOCK, cols, BLOCK)


def _scale(largest):
    """The scale of a block whose largest magnitude is given: at least the smallest normal float."""
    s = largest / torch.full_like(largest, E4M3_MAX)
    return torch.clamp_min(s, torch.finfo(torch.float32).tiny)


def _quantized_weight(w):
    t = _tiles(w)
    scales = _scale(t.abs().amax(dim=(1, 3)))
    q = (t / scales[:, None, :, None]).reshape(t.shape[0] * BLOCK, -1)[:w.shape[0], :w.shape[1]]
    return q.contiguous().to(torch.float8_e4m3fn), scales


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    kind, t, n = case["kind"], case["t"], case["n"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case)
    if kind.startswith("norm"):
        # a residual stream: each channel with its own mean and spread
        spread = 0.5 + torch.rand(n, generator=g, device=DEV)
        shift = torch.randn(n, generator=g, device=DEV) * 0.3
        s["x"] = (torch.randn(t, n, generator=g, device=DEV) * spread + shift).to(dt)
        s["w"] = (1 + torch.randn(n, generator=g, device=DEV) * 0.1).to(dt)
        s["b"] = normal(n, std=0.1)
        if kind == "norm_bwd":
            y = _plain_norm({**s, "eps": 1e-5})
            s["mean"], s["rstd"] = y["mean"], y["rstd"]
            s["dy"] = normal(t, n)
            s["r"] = normal(t, n) if case["residual"] else None
        return s
    k = case["k"]
    # activations behind a norm: a few channels are larger than the others
    s["x"] = (torch.randn(t, k, generator=g, device=DEV) *
              (0.5 + torch.rand(k, generator=g, device=DEV) ** 4 * 4)).to(dt)
    if kind == "block":
        s["w"], s["scales"] = _quantized_weight(normal(n, k, std=k ** -0.5, dtype=torch.float32))
        s["b"] = normal(n, std=0.1) if case["bias"] else None
        s["r"] = normal(t, n) if case["residual"] else None
        return s
    s["w"] = normal(2 * n, k, std=k ** -0.5)
    s["b"] = normal(2 * n, std=0.1) if case["bias"] else None
    if kind == "gated_bwd":
        z = s["x"] @ s["w"].t()
        s["z"] = z + s["b"] if case["bias"] else z
        s["dy"] = normal(t, n)
    return s


# ---- one pass ---------------------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return _PLAIN[s["kind"]](s)


def _own(s):
    import precision_gemm_gb300 as pg
    kind = s["kind"]
    if kind == "norm":
        y, mean, rstd = pg.layer_norm(s["x"], s["w"], s["b"], s["eps"], stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "norm_bwd":
        dx, dw, db = pg.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], residual=s["r"])
        return {"dx": dx, "dw": dw, "db": db}
    if kind == "gated":
        if s["keep"]:
            y, z = pg.gated_linear(s["x"], s["w"], s["b"], s["act"], preact=True)
            return {"y": y, "z": z}
        return {"y": pg.gated_linear(s["x"], s["w"], s["b"], s["act"])}
    if kind == "gated_bwd":
        dx, dw, db = pg.gated_linear_backward(s["dy"], s["x"], s["w"], s["z"], s["act"], bias=s["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    return pg.block_linear(s["x"], s["w"], s["scales"], s["b"], s["act"], residual=s["r"])


# ---- the plain forms: elementary operations in 32 bits -----------------------------------


def _act(z, name):
    if name == "relu":
        return torch.clamp_min(z, 0.0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * (0.5 ** 0.5)))
    return z


def _dact(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * (0.5 ** 0.5))) + z * torch.exp(-0.5 * z * z) * ((2 * math.pi) ** -0.5)
    return torch.ones_like(z)


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + s["eps"])
    y = c * rstd * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_bwd(s):
    dt = s["x"].dtype
    dy = s["dy"].float()
    h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return {"dx": dx.to(dt), "dw": (dy * h).sum(0).to(dt), "db": dy.sum(0).to(dt)}


def _plain_gated(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    g, u = z[:, :s["n"]], z[:, s["n"]:]
    y = {"y": (_act(g, s["act"]) * u).to(s["x"].dtype)}
    if s["keep"]:
        y["z"] = z.to(s["x"].dtype)
    return y


def _plain_gated_bwd(s):
    dt, n = s["x"].dtype, s["n"]
    g, u = s["z"][:, :n].float(), s["z"][:, n:].float()
    dy = s["dy"].float()
    dz = torch.cat([dy * u * _dact(g, s["act"]), dy * _act(g, s["act"])], dim=1)
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt),
            "db": dz.sum(0).to(dt) if s["bias"] else None}


def _plain_block(s):
    x = s["x"].float()
    t, k = x.shape
    cols = -(-k // BLOCK)
    full = x.new_zeros(t, cols * BLOCK)
    full[:, :k] = x
    full = full.view(t, cols, BLOCK)
    scale = _scale(full.abs().amax(dim=2, keepdim=True))
    x = ((full / scale).to(torch.float8_e4m3fn).float() * scale).view(t, cols * BLOCK)[:, :k]
    spread = s["scales"].repeat_interleave(BLOCK, 0)[:s["n"]].repeat_interleave(BLOCK, 1)[:, :k]
    y = x @ (s["w"].float() * spread).t()
    if s["b"] is not None:
        y = y + s["b"].float()
    y = _act(y, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["x"].dtype)


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "gated": _plain_gated, "gated_bwd": _plain_gated_bwd,
          "block": _plain_block}


# ---- the definitions in 64 bits -------------------------------------------------------------


def _f64(z, name):
    """An activation in 64 bits, from the functions' definitions."""
    if name == "relu":
        return torch.relu(z)
    if name == "silu":
        return z * torch.special.expit(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z


def _to_e4m3(v):
    """v (64 bits, at most 448) rounded to the nearest of e4m3's values, ties to even: three bits behind
    the leading one, steps of 2^-9 below 2^-6."""
    exponent = torch.frexp(v)[1] - 1
    step = torch.exp2(exponent.clamp_min(-6).double() - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    kind = case["kind"]
    if kind == "norm":
        var, mean = torch.var_mean(d["x"], dim=1, correction=0)
        rstd = torch.rsqrt(var + case["eps"])
        y = torch.einsum("tn,t,n->tn", d["x"] - mean[:, None], rstd, d["w"]) + d["b"]
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "norm_bwd":
        x, w, b = (d[k].detach().requires_grad_(True) for k in ("x", "w", "b"))
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        y = (x - mean) * torch.rsqrt(var + 1e-5) * w + b
        dx, dw, db = torch.autograd.grad(y, (x, w, b), d["dy"])
        return {"dx": dx if d["r"] is None else dx + d["r"], "dw": dw, "db": db}
    n = case["n"]
    if kind == "gated":
        z = torch.einsum("tk,nk->tn", d["x"], d["w"])
        z = z if d["b"] is None else z + d["b"]
        y = {"y": _f64(z[:, :n], case["act"]) * z[:, n:]}
        return {**y, "z": z} if case["keep"] else y
    if kind == "gated_bwd":
        z = d["z"].detach().requires_grad_(True)
        dz = torch.autograd.grad(_f64(z[:, :n], case["act"]) * z[:, n:], z, d["dy"])[0]
        return {"dx": torch.einsum("tn,nk->tk", dz, d["w"]), "dw": torch.einsum("tn,tk->nk", dz, d["x"]),
                "db": torch.einsum("tn->n", dz) if case["bias"] else None}
    y = torch.zeros(case["t"], n, dtype=torch.float64, device=DEV)
    for j, at in enumerate(range(0, case["k"], BLOCK)):
        x = d["x"][:, at:at + BLOCK]
        # a scale is a float32 number, and so is the quotient that is rounded to e4m3: of bfloat16 values it often
        # falls between two of e4m3's, and a quotient of more bits would fall to one side
        scale = (x.abs().amax(1, keepdim=True) / E4M3_MAX).float().double().clamp_min(2.0 ** -126)
        x = _to_e4m3((x / scale).float().double())
        w = d["w"][:, at:at + BLOCK] * d["scales"][torch.arange(n, device=DEV) // BLOCK, j][:, None]
        y += scale * (x @ w.t())
    y = _f64(y if d["b"] is None else y + d["b"], case["act"])
    return y if d["r"] is None else y + d["r"]


# ---- what a pass cannot do without ------------------------------------------------------------


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    kind, t, n = case["kind"], case["t"], case["n"]
    if kind == "norm":
        return {"bytes": size * (2 * t * n + 2 * n) + 8 * t, "flops": 8 * t * n}
    if kind == "norm_bwd":
        return {"bytes": size * ((4 if case["residual"] else 3) * t * n + 3 * n) + 8 * t, "flops": 14 * t * n}
    k = case["k"]
    if kind == "gated":
        return {"bytes": size * (t * k + 2 * n * k + t * n * (3 if case["keep"] else 1) +
                                 (2 * n if case["bias"] else 0)), "flops": 4 * t * n * k}
    if kind == "gated_bwd":
        return {"bytes": size * (3 * t * n + 2 * t * k + 4 * n * k + (2 * n if case["bias"] else 0)),
                "flops": 8 * t * n * k}
    scales = 4 * -(-n // BLOCK) * -(-k // BLOCK)
    return {"bytes": size * (t * k + t * n * (2 if case["residual"] else 1) + (n if case["bias"] else 0)) + n * k +
            scales, "flops": 2 * t * n * k}
