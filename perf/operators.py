"""Measured work of the feed-forward operators: linear layers with a fused
epilogue, routing to experts, and the experts' products, in both directions.

A case is one pass through one operator.  `own` selects who computes it: the
operators' plain form (elementary torch operations in 32 bits, rounded once at
the end) or this package's public calls.  `exact` is the same pass from the
definitions in 64 bits.

Kinds of a case:
  linear        y = act(x w^T + b) + r
  linear_bwd    (dx, dw, db) of act(x w^T + b) for dy, with the saved x w^T + b
  route         top-k experts and weights of each token, and the experts' row lists
  route_bwd     gradient of the logits for a gradient of the routing weights
  experts       the experts' row lists, then h = act(x[token] w[e]^T + b[e]) per (token, expert) row
  experts_ffn   a whole expert feed-forward: up product, down product, weighted sum per token
  experts_bwd   (dx, dw, db) of `experts`, with the saved pre-activation
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # One token through a square projection: a decoding step of a dense layer, where the weights' read time is all.
        {"name": "linear decode bf16", "kind": "linear", "t": 1, "n": 4096, "k": 4096, "dtype": "bf16", "act": "none",
         "bias": True, "residual": True},
        # A handful of drafted or batched tokens through an up projection whose weights are kept in float32.
        {"name": "linear few tokens f32", "kind": "linear", "t": 5, "n": 8192, "k": 2048, "dtype": "f32", "act": "silu",
         "bias": True, "residual": False},
        # A prompt of 2048 tokens through the up projection of a feed-forward block.
        {"name": "linear prefill bf16", "kind": "linear", "t": 2048, "n": 8192, "k": 4096, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False},
        # The repository's ragged sizes (3000 x 1500 x 777): no extent is a multiple of a tile, rows are not 16-byte aligned.
        {"name": "linear ragged f32", "kind": "linear", "t": 1500, "n": 3000, "k": 777, "dtype": "f32", "act": "silu",
         "bias": True, "residual": True},
        # A training step's backward pass through an up projection, 8192 tokens.
        {"name": "linear backward bf16", "kind": "linear_bwd", "t": 8192, "n": 8192, "k": 2048, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False},
        # The backward pass at the odd sizes 1300 x 1000 x 1500, all in float32.
        {"name": "linear backward f32", "kind": "linear_bwd", "t": 1300, "n": 1000, "k": 1500, "dtype": "f32",
         "act": "silu", "bias": True, "residual": False},
        # Routing of eight tokens that decode together: the latency of two small steps.
        {"name": "route decode", "kind": "route", "t": 8, "experts": 64, "top": 6, "score": "softmax", "bias": False,
         "groups": 1, "group_top": 1, "renorm": True, "dtype": "bf16", "mask": False},
        # Routing of a long prompt: sigmoid scores, balance bias, 4 of 8 groups, some padded tokens.
        {"name": "route prefill", "kind": "route", "t": 16384, "experts": 256, "top": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "group_top": 4, "renorm": True, "dtype": "f32", "mask": True},
        # The router's backward pass over a large training batch.
        {"name": "route backward", "kind": "route_bwd", "t": 65536, "experts": 128, "top": 8, "score": "softmax",
         "bias": False, "groups": 1, "group_top": 1, "renorm": True, "dtype": "f32", "mask": False},
        # Four tokens that decode together through a float32 expert feed-forward: most experts are empty.
        {"name": "experts decode f32", "kind": "experts_ffn", "t": 4, "experts": 64, "top": 8, "n": 1024, "k": 2048,
         "dtype": "f32", "act": "silu"},
        # A prompt of 8192 tokens through the up product of 64 experts with uneven loads.
        {"name": "experts prefill bf16", "kind": "experts", "t": 8192, "experts": 64, "top": 8, "n": 1024, "k": 2048,
         "dtype": "bf16", "act": "gelu"},
        # The same layer's backward pass on 4096 tokens.
        {"name": "experts backward bf16", "kind": "experts_bwd", "t": 4096, "experts": 64, "top": 8, "n": 1024,
         "k": 2048, "dtype": "bf16", "act": "gelu"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _extent(rng, lo, hi):
    """A feature count: half of the draws multiples of 64, the others as they come, odd ones among them."""
    v = _log(rng, lo, hi)
    return max(lo, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear_bwd", "route", "route_bwd", "experts", "experts_ffn", "experts_bwd"])
    act = rng.choice(["none", "relu", "silu", "gelu"])
    dtype = rng.choice(["bf16", "f32"])
    if kind in ("linear", "linear_bwd"):
        return {"kind": kind, "t": _log(rng, 1 if kind == "linear" else 64, 8192), "n": _extent(rng, 64, 8192),
                "k": _extent(rng, 64, 4096 if kind == "linear" else 2048), "dtype": dtype, "act": act,
                "bias": rng.random() < 0.7, "residual": kind == "linear" and rng.random() < 0.5}
    if kind in ("route", "route_bwd"):
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256])
        top = rng.randint(1, 8)
        groups = rng.choice([1, 1, 4]) if top <= experts // 4 else 1
        score = rng.choice(["softmax", "sigmoid"])
        # (a single weight that is renormalised is 1 and has no gradient)
        renorm = rng.random() < 0.7 and (top > 1 or kind == "route")
        return {"kind": kind, "t": _log(rng, 1, 65536), "experts": experts, "top": top, "score": score,
                "bias": rng.random() < 0.5, "groups": groups, "group_top": 2 if groups > 1 else 1,
                "renorm": renorm, "dtype": dtype, "mask": rng.random() < 0.3}
    experts = rng.choice([8, 16, 60, 64])
    return {"kind": kind, "t": _log(rng, 1 if kind != "experts_bwd" else 64, 4096), "experts": experts,
            "top": rng.randint(1, 8), "n": _extent(rng, 64, 1024), "k": _extent(rng, 64, 2048),
            "dtype": "f32" if kind == "experts_ffn" else dtype, "act": act}


# ---- inputs ---------------------------------------------------------------------------


def _lists(experts, count):
    """The experts' row lists of (token, choice) pairs: counts, offsets, the pair of
    each row (pairs of one expert in their order) and the row of each pair."""
    flat = experts.reshape(-1)
    kept = torch.where(flat < 0, count, flat)
    rows = torch.argsort(kept, stable=True)
    counts = torch.bincount(kept, minlength=count + 1)[:count]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    valid = torch.arange(flat.numel(), device=flat.device) < offsets[-1]
    slots = torch.empty_like(rows)
    slots[rows] = torch.arange(flat.numel(), device=flat.device)
    slots = torch.where(flat < 0, -1, slots)
    rows = torch.where(valid, rows, -1)
    return tuple(v.to(torch.int32) for v in (counts, offsets, rows, slots.reshape(experts.shape)))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    kind, t = case["kind"], case["t"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case)
    if kind.startswith("linear"):
        n, k = case["n"], case["k"]
        s["x"] = normal(t, k)
        s["w"] = normal(n, k, std=k ** -0.5)
        s["b"] = normal(n, std=0.1) if case["bias"] else None
        s["r"] = normal(t, n) if case["residual"] else None
        if kind == "linear_bwd":
            z = s["x"] @ s["w"].t()
            s["z"] = z + s["b"] if case["bias"] else z
            s["dy"] = normal(t, n)
        return s
    e, top = case["experts"], case["top"]
    if kind.startswith("route"):
        # logits of a trained router: spread over tokens, and some experts preferred throughout
        s["logits"] = (torch.randn(t, e, generator=g, device=DEV) * 1.5 +
                       torch.randn(e, generator=g, device=DEV) * 0.5).to(dt)
        s["balance"] = normal(e, std=0.05, dtype=torch.float32) if case["bias"] else None
        s["valid"] = torch.rand(t, generator=g, device=DEV) < 0.9 if case["mask"] else None
        if kind == "route_bwd":
            s["ids"] = _plain_route(s)[1]
            s["dweights"] = normal(t, top, dtype=torch.float32)
        return s
    n, k = case["n"], case["k"]
    scores = torch.rand(t, e, generator=g, device=DEV) + torch.rand(e, generator=g, device=DEV) * 0.5
    s["ids"] = torch.topk(scores, top, dim=1).indices.to(torch.int32)
    s["cap"] = int(torch.bincount(s["ids"].reshape(-1).long(), minlength=e).max())  # the plain form's padded length
    s["x"] = normal(t, k)
    s["w"] = normal(e, n, k, std=k ** -0.5)
    s["b"] = normal(e, n, std=0.1)
    if kind == "experts_ffn":
        s["w2"] = normal(e, k, n, std=n ** -0.5)
        s["weights"] = torch.softmax(torch.randn(t, top, generator=g, device=DEV), dim=1)
        s["r"] = normal(t, k)
    if kind == "experts_bwd":
        s["lists"] = _lists(s["ids"], e)
        h = torch.cat([s["x"][r.long() // top] @ s["w"][i].t() + s["b"][i]
                       for i, r in enumerate(torch.split(s["lists"][2], s["lists"][0].tolist()))])
        s["z"] = h
        s["dh"] = normal(t * top, n)
    return s


# ---- one pass ---------------------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    return _PLAIN[s["kind"]](s)


def _own(s):
    import precision_gemm_gb300 as pg
    kind = s["kind"]
    if kind == "linear":
        return pg.linear(s["x"], s["w"], s["b"], s["act"], residual=s["r"])
    if kind == "linear_bwd":
        dx, dw, db = pg.linear_backward(s["dy"], s["x"], s["w"], s["act"], preact=s["z"], bias=s["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    if kind == "route":
        weights, ids = pg.route(s["logits"], s["top"], s["score"], bias=s["balance"], groups=s["groups"],
                                group_top=s["group_top"], renormalize=s["renorm"], mask=s["valid"])
        plan = pg.expert_plan(ids, s["experts"])
        return {"weights": weights, "ids": ids, "counts": plan.counts, "offsets": plan.offsets, "rows": plan.rows,
                "slots": plan.slots}
    if kind == "route_bwd":
        return pg.route_backward(s["dweights"], s["logits"], s["ids"], s["score"], renormalize=s["renorm"])
    if kind == "experts":
        plan = pg.expert_plan(s["ids"], s["experts"])
        h = pg.expert_linear(s["x"], s["w"], plan, s["b"], s["act"], gather=True)
        return {"h": h, "counts": plan.counts}
    if kind == "experts_ffn":
        plan = pg.expert_plan(s["ids"], s["experts"])
        h = pg.expert_linear(s["x"], s["w"], plan, s["b"], s["act"], gather=True)
        o = pg.expert_linear(h, s["w2"], plan)
        return pg.expert_combine(o, plan, s["weights"], residual=s["r"])
    plan = pg.ExpertPlan(*s["lists"])
    dx, dw, db = pg.expert_linear_backward(s["dh"], s["x"], s["w"], plan, s["act"], preact=s["z"], bias=True,
                                           gather=True)
    return {"dx": dx, "dw": dw, "db": db}


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


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        y = y + s["b"].float()
    y = _act(y, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["x"].dtype)


def _plain_linear_bwd(s):
    dt = s["x"].dtype
    dz = s["dy"].float() * _dact(s["z"].float(), s["act"])
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt),
            "db": dz.sum(0).to(dt) if s["bias"] else None}


def _scores(logits, score):
    """Scores in 32 bits; a softmax row's sum is taken in 64 bits, so that it does not depend on an order."""
    x = logits.float()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    ex = torch.exp(x - x.max(dim=1, keepdim=True).values)
    return ex / ex.sum(dim=1, keepdim=True, dtype=torch.float64).float()


def _plain_route(s):
    p = _scores(s["logits"], s["score"])
    choice = p if s["balance"] is None else p + s["balance"]
    t, e = choice.shape
    if s["groups"] > 1:
        per = choice.view(t, s["groups"], e // s["groups"])
        best = torch.sort(per, dim=2, descending=True).values[:, :, :2].sum(2)
        # descending and stable: equal values keep the lower index first
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["group_top"]]
        inside = torch.zeros(t, s["groups"], dtype=torch.bool, device=p.device).scatter_(1, kept, True)
        choice = torch.where(inside.repeat_interleave(e // s["groups"], 1), choice, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :s["top"]]
    w = torch.gather(p, 1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if s["valid"] is not None:
        w = torch.where(s["valid"][:, None], w, 0.0)
        ids = torch.where(s["valid"][:, None], ids, -1)
    return w, ids.to(torch.int32)


def _plain_routing(s):
    weights, ids = _plain_route(s)
    counts, offsets, rows, slots = _lists(ids, s["experts"])
    return {"weights": weights, "ids": ids, "counts": counts, "offsets": offsets, "rows": rows, "slots": slots}


def _plain_route_bwd(s):
    p = _scores(s["logits"], s["score"])
    ids = s["ids"].long()
    held = (ids >= 0).float()
    at = ids.clamp_min(0)
    q = torch.gather(p, 1, at) * held
    dw = s["dweights"] * held
    if s["renorm"]:
        total = q.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        dq = (dw - (dw * q).sum(1, keepdim=True) / total) / total
    else:
        dq = dw
    dp = torch.zeros_like(p).scatter_add_(1, at, dq * held)
    if s["score"] == "sigmoid":
        dx = dp * p * (1 - p)
    else:
        dx = p * (dp - (dp * p).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


def _places(lists, ids):
    """Of each row: its expert, its place in the expert's list, its token."""
    counts, offsets, rows, _ = (v.long() for v in lists)
    expert = ids.reshape(-1).long()[rows]
    return expert, torch.arange(rows.numel(), device=rows.device) - offsets[expert], rows // ids.shape[1]


def _product(rows, w, expert, place, cap):
    """rows[r] @ w[expert[r]]^T: few rows gather their experts' matrices, many are laid out per expert."""
    if rows.shape[0] <= w.shape[0]:
        return torch.bmm(w[expert].float(), rows[:, :, None])[:, :, 0]
    x = rows.new_zeros(w.shape[0], cap, rows.shape[1])
    x[expert, place] = rows
    return torch.bmm(x, w.float().transpose(1, 2))[expert, place]


def _plain_experts(s):
    lists = _lists(s["ids"], s["experts"])
    expert, place, token = _places(lists, s["ids"])
    z = _product(s["x"][token].float(), s["w"], expert, place, s["cap"]) + s["b"].float()[expert]
    return {"h": _act(z, s["act"]).to(s["x"].dtype), "counts": lists[0]}


def _plain_experts_ffn(s):
    lists = _lists(s["ids"], s["experts"])
    expert, place, token = _places(lists, s["ids"])
    z = _product(s["x"][token].float(), s["w"], expert, place, s["cap"]) + s["b"].float()[expert]
    o = _product(_act(z, s["act"]), s["w2"], expert, place, s["cap"])
    y = (o[lists[3].long()] * s["weights"][:, :, None]).sum(1) + s["r"].float()
    return y.to(s["x"].dtype)


def _plain_experts_bwd(s):
    expert, place, token = _places(s["lists"], s["ids"])
    dt, w = s["x"].dtype, s["w"]
    dz = s["dh"].float() * _dact(s["z"].float(), s["act"])
    cap = s["cap"]
    dzp = dz.new_zeros(w.shape[0], cap, dz.shape[1])
    dzp[expert, place] = dz
    xp = dz.new_zeros(w.shape[0], cap, w.shape[2])
    xp[expert, place] = s["x"][token].float()
    rows = torch.bmm(dzp, w.float())[expert, place]
    return {"dx": rows[s["lists"][3].long()].sum(1).to(dt), "dw": torch.bmm(dzp.transpose(1, 2), xp).to(dt),
            "db": dzp.sum(1).to(dt)}


_PLAIN = {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "route": _plain_routing,
          "route_bwd": _plain_route_bwd, "experts": _plain_experts, "experts_ffn": _plain_experts_ffn,
          "experts_bwd": _plain_experts_bwd}


# ---- the definitions in 64 bits -------------------------------------------------------------


def _f64(z, name):
    """Activation and derivative in 64 bits, from the functions' definitions."""
    if name == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros_like(z))
    if name == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    kind = case["kind"]
    if kind == "linear":
        z = torch.einsum("tk,nk->tn", d["x"], d["w"])
        z = z if d["b"] is None else z + d["b"]
        y = _f64(z, case["act"])[0]
        return y if d["r"] is None else y + d["r"]
    if kind == "linear_bwd":
        dz = d["dy"] * _f64(d["z"], case["act"])[1]
        return {"dx": torch.einsum("tn,nk->tk", dz, d["w"]), "dw": torch.einsum("tn,tk->nk", dz, d["x"]),
                "db": torch.einsum("tn->n", dz) if case["bias"] else None}
    if kind in ("route", "route_bwd"):
        x = d["logits"]
        p = torch.special.expit(x) if case["score"] == "sigmoid" else torch.softmax(x, dim=1)
        if kind == "route":
            # the weights at the experts that 32-bit scores choose: the choice itself is no computed number
            ids = _plain_route(s)[1].long()
            w = torch.take_along_dim(p, ids.clamp_min(0), 1)
            w = w / w.sum(1, keepdim=True) if case["renorm"] else w
            return {"weights": torch.where(ids >= 0, w, 0.0), "ids": None, "counts": None, "offsets": None,
                    "rows": None, "slots": None}
        x = x.detach().requires_grad_(True)
        p = torch.special.expit(x) if case["score"] == "sigmoid" else torch.softmax(x, dim=1)
        ids = s["ids"].long()
        w = torch.take_along_dim(p, ids.clamp_min(0), 1) * (ids >= 0)
        if case["renorm"]:
            w = w / torch.where(w.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), 1.0)
        return torch.autograd.grad((w * d["dweights"]).sum(), x)[0]
    e, top = case["experts"], case["top"]
    flat = s["ids"].reshape(-1)
    members = [torch.nonzero(flat == i)[:, 0] for i in range(e)]
    if kind == "experts":
        h = [_f64(d["x"][m // top] @ d["w"][i].t() + d["b"][i], case["act"])[0] for i, m in enumerate(members)]
        return {"h": torch.cat(h), "counts": None}
    if kind == "experts_ffn":
        y = d["r"].clone()
        share = d["weights"].reshape(-1)
        for i, m in enumerate(members):
            h = _f64(d["x"][m // top] @ d["w"][i].t() + d["b"][i], case["act"])[0]
            y.index_add_(0, m // top, share[m, None] * (h @ d["w2"][i].t()))
        return y
    dz = d["dh"] * _f64(d["z"], case["act"])[1]
    dx, dw, db, at = torch.zeros_like(d["x"]), torch.zeros_like(d["w"]), torch.zeros_like(d["b"]), 0
    for i, m in enumerate(members):
        part = dz[at:at + m.numel()]
        at += m.numel()
        dx.index_add_(0, m // top, part @ d["w"][i])
        dw[i] = part.t() @ d["x"][m // top]
        db[i] = part.sum(0)
    return {"dx": dx, "dw": dw, "db": db}


# ---- what a pass cannot do without ------------------------------------------------------------


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    kind, t = case["kind"], case["t"]
    if kind == "linear":
        n, k = case["n"], case["k"]
        return {"bytes": size * (t * k + n * k + t * n * (2 if case["residual"] else 1) + (n if case["bias"] else 0)),
                "flops": 2 * t * n * k}
    if kind == "linear_bwd":
        n, k = case["n"], case["k"]
        gated = 2 if case["act"] != "none" else 1
        return {"bytes": size * (gated * t * n + 2 * (t * k + n * k) + (n if case["bias"] else 0)),
                "flops": 4 * t * n * k}
    e, top = case["experts"], case["top"]
    if kind == "route":
        return {"bytes": size * t * e + 16 * t * top, "flops": 4 * t * e}
    if kind == "route_bwd":
        return {"bytes": 2 * size * t * e + 8 * t * top, "flops": 8 * t * e}
    n, k, rows = case["n"], case["k"], t * top
    used = e * (1 - (1 - 1 / e) ** rows)  # experts that a token reaches, of even chances
    if kind == "experts":
        return {"bytes": size * (t * k + rows * n + used * (n * k + n)) + 4 * rows, "flops": 2 * rows * n * k}
    if kind == "experts_ffn":
        return {"bytes": size * (3 * t * k + used * (2 * n * k + n)) + 8 * rows, "flops": 4 * rows * n * k}
    gated = 2 if case["act"] != "none" else 1
    return {"bytes": size * (2 * t * k + gated * rows * n + used * n * k + e * (n * k + n)) + 8 * rows,
            "flops": 4 * rows * n * k}
