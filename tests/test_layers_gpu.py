"""Linear layers and the experts' products against their definitions in 64 bits:
sizes from zero and one to several tiles, odd extents, strided and unaligned rows,
empty experts, pairs of no expert, every activation, both types and directions."""
import math

import pytest
import torch

import precision_gemm_gb300 as pg
from tests import _layers_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
IDS = {torch.float32: "f32", torch.bfloat16: "bf16"}


@pytest.fixture(autouse=True)
def _healthy():
    pg.load_library()
    pg.device_status()
    yield
    assert pg.device_status() == 0


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _draw(g, dtype, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _strided(x, pad, offset=0):
    """A CUDA copy of matrix x whose rows are pad elements apart more than they are
    long, its first element `offset` elements into the storage; the gaps hold NaN."""
    r, c = x.shape
    buf = torch.full((offset + r * (c + pad),), math.nan, dtype=x.dtype, device="cuda")
    view = buf[offset:].view(r, c + pad)[:, :c] if r else buf[offset:].view(0, c + pad)[:, :c]
    view.copy_(x)
    return view


SIZES = [(1, 1, 1), (1, 130, 3), (2, 4096, 512), (3, 64, 64), (5, 1000, 777), (8, 96, 2048), (17, 257, 129),
         (33, 640, 256), (64, 128, 64), (130, 300, 777), (257, 513, 1000), (300, 256, 65), (1500, 300, 777)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k", SIZES)
def test_linear(dtype, t, n, k):
    g = _gen(t * 7 + n * 3 + k)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, n, k, std=k ** -0.5)
    b, r = _draw(g, dtype, n), _draw(g, dtype, t, n)
    name = R.ACTS[(t + n + k) % 5]
    y, z = pg.linear(x.cuda(), w.cuda(), b.cuda(), name, r.cuda(), preact=True)
    want, wz, den = R.linear(x, w, b, name, r)
    R.close(y, want, den, dtype)
    R.close(z, wz, den, dtype)
    y = pg.linear(x.cuda(), w.cuda())
    want, _, den = R.linear(x, w, None, "none", None)
    R.close(y, want, den, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("t", [4, 200])
def test_linear_activations_over_their_range(dtype, name, t):
    # pre-activations from -12 to 12: both tails of every activation, and its zero
    n, k = 192, 32
    g = _gen(5)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, n, k, std=k ** -0.5)
    b = torch.linspace(-12, 12, n).to(dtype)
    x[0] = 0
    y = pg.linear(x.cuda(), w.cuda(), b.cuda(), name)
    want, _, den = R.linear(x, w, b, name, None)
    R.close(y, want, den, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k,pad,offset", [(6, 70, 100, 3, 1), (140, 200, 136, 5, 3), (140, 200, 136, 8, 8),
                                              (300, 130, 64, 1, 0), (1, 64, 72, 7, 2)])
def test_linear_strides_and_alignment(dtype, t, n, k, pad, offset):
    g = _gen(t + pad)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, n, k, std=k ** -0.5)
    b, r = _draw(g, dtype, n), _draw(g, dtype, t, n)
    out = _strided(torch.zeros(t, n, dtype=dtype), pad, offset)
    got = pg.linear(_strided(x, pad, offset), _strided(w, pad, offset), b.cuda(), "silu", _strided(r, pad, offset),
                    out=out)
    assert got is out
    want, _, den = R.linear(x, w, b, "silu", r)
    R.close(out, want, den, dtype)
    gaps = out.as_strided((t, pad), (n + pad, 1), offset + n)[:t - 1]
    assert torch.isnan(gaps).all()  # nothing between the rows was written
    # residual and result in one tensor
    both = r.cuda()
    pg.linear(x.cuda(), w.cuda(), b.cuda(), "gelu", both, out=both)
    want, _, den = R.linear(x, w, b, "gelu", r)
    R.close(both, want, den, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_linear_empty_extents_and_leading_dimensions(dtype):
    g = _gen(1)
    b, r = _draw(g, dtype, 9), _draw(g, dtype, 4, 9)
    y = pg.linear(torch.empty(4, 0, dtype=dtype, device="cuda"), torch.empty(9, 0, dtype=dtype, device="cuda"),
                  b.cuda(), "silu", r.cuda())
    want, _, den = R.linear(torch.zeros(4, 0), torch.zeros(9, 0), b, "silu", r)
    R.close(y, want, den, dtype)
    assert pg.linear(torch.empty(0, 5, dtype=dtype, device="cuda"),
                     torch.empty(9, 5, dtype=dtype, device="cuda")).shape == (0, 9)
    x, w = _draw(g, dtype, 2, 3, 40), _draw(g, dtype, 24, 40)
    y, z = pg.linear(x.cuda(), w.cuda(), preact=True)
    assert y.shape == z.shape == (2, 3, 24)
    want, _, den = R.linear(x.view(6, 40), w, None, "none", None)
    R.close(y.view(6, 24), want, den, dtype)
    dx, dw, db = pg.linear_backward(torch.empty(0, 9, dtype=dtype, device="cuda"),
                                    torch.empty(0, 5, dtype=dtype, device="cuda"),
                                    torch.empty(9, 5, dtype=dtype, device="cuda"))
    assert dx.shape == (0, 5) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t", [3, 150])
def test_linear_infinities_and_nan_stay_in_their_rows(dtype, t):
    n, k = 140, 200
    g = _gen(3)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, n, k)
    x[1, 7], x[2, 11] = math.inf, math.nan
    y = pg.linear(x.cuda(), w.cuda()).cpu()
    want = (x.double() @ w.double().t())
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(y), finite)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y[1].double(), want[1])  # signed infinities
    assert finite[0].all() and not finite[1].any() and torch.isnan(want[2]).all()


@pytest.mark.parametrize("t", [4, 300])
def test_linear_float32_is_not_tf32(t):
    """The 2-norm of the error stays at FP32's: the longest run of additions whose results
    are truncated is 32 (2^-24 of the sum each, all one way), doubled for the rest."""
    n, k = 512, 4096
    g = _gen(t)
    x, w = _draw(g, torch.float32, t, k), _draw(g, torch.float32, n, k, std=k ** -0.5)
    y = pg.linear(x.cuda(), w.cuda()).double().cpu()
    want = x.double() @ w.double().t()
    assert float((y - want).norm() / want.norm()) < 64 * 2.0 ** -24


def _inner(dtype, name):
    """The rounding of dz to bfloat16 before the products (exact when dz is dy)."""
    return R.HALF if dtype == torch.bfloat16 and name != "none" else 0.0


def _check_backward(got, want, den, dtype, name):
    for i, (a, b, d) in enumerate(zip(got, want, den)):
        # the bias gradient sums unrounded terms
        R.close(a, b, d, dtype, slope=1.0, inner=_inner(dtype, name) if i < 2 else 0.0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 70, 130), (5, 64, 64), (63, 65, 66), (130, 300, 77), (257, 130, 200),
                                   (640, 256, 384), (1300, 100, 150)])
def test_linear_backward(dtype, t, n, k):
    g = _gen(t + n + k)
    name = R.ACTS[(t + n + k) % 5]
    x, w, dy = _draw(g, dtype, t, k), _draw(g, dtype, n, k, std=k ** -0.5), _draw(g, dtype, t, n)
    z = _draw(g, dtype, t, n, std=2.0)
    got = pg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), name, z.cuda())
    want, den = R.linear_backward(dy, x, w, name, z)
    _check_backward(got, want, den, dtype, name)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_linear_backward_strides_and_skipped_gradients(dtype, name):
    t, n, k = 150, 170, 90
    g = _gen(8)
    x, w, dy = _draw(g, dtype, t, k), _draw(g, dtype, n, k, std=k ** -0.5), _draw(g, dtype, t, n)
    z = _draw(g, dtype, t, n)
    args = (_strided(dy, 3, 1), _strided(x, 5, 3), _strided(w, 1, 7), name, _strided(z, 9, 5))
    want, den = R.linear_backward(dy, x, w, name, z)
    _check_backward(pg.linear_backward(*args), want, den, dtype, name)
    whole = pg.linear_backward(*args)
    dx, dw, db = pg.linear_backward(*args, need_dw=False, bias=False)
    assert dw is None and db is None and torch.equal(dx, whole[0])
    dx, dw, db = pg.linear_backward(*args, need_dx=False)
    assert dx is None and torch.equal(dw, whole[1]) and torch.equal(db, whole[2])


@pytest.mark.parametrize("name", R.ACTS)
def test_linear_backward_against_differences(name):
    """Directional differences of the 64-bit layer around the point, step 1e-5: their own
    error is of order 1e-10, the FP32 gradient's 1e-6 of the terms' sizes."""
    t, n, k = 40, 50, 60
    g = _gen(11)
    x, w, b = (torch.randn(*s, generator=g) for s in ((t, k), (n, k), (n,)))
    x = torch.where(x.abs() < 1e-2, torch.full_like(x, 0.1), x)
    w = w * k ** -0.5
    dy = torch.randn(t, n, generator=g)
    y, z = pg.linear(x.cuda(), w.cuda(), b.cuda(), name, preact=True)
    dx, dw, db = pg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), name, z)

    def loss(x, w, b):
        return float((R.linear(x, w, b, name, None)[0] * dy.double()).sum())

    h = 1e-5
    for i, (v, grad) in enumerate(((x, dx), (w, dw), (b, db))):
        u = torch.randn(v.shape, generator=g, dtype=torch.float64)
        at = [x.double(), w.double(), b.double()]
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * u, at[i] - h * u
        diff = (loss(*up) - loss(*down)) / (2 * h)
        scale = float((grad.double().cpu().abs() * u.abs()).sum())
        assert abs(diff - float((grad.double().cpu() * u).sum())) <= 2e-5 * scale, (name, i)


# ---- experts -----------------------------------------------------------------------


def _ids(g, t, top, e, kind):
    if kind == "even":
        return torch.stack([torch.randperm(e, generator=g)[:top] for _ in range(t)]).to(torch.int32)
    if kind == "one":  # every pair to one expert, the others empty
        return torch.full((t, top), e // 2, dtype=torch.int32)
    ids = torch.randint(0, max(1, e // 2), (t, top), generator=g, dtype=torch.int32)  # half of the experts empty
    if kind == "dropped":
        drop = torch.rand(t, top, generator=g) < 0.3
        ids = torch.where(drop, torch.where(torch.rand(t, top, generator=g) < 0.5, -1, e + 3).to(torch.int32), ids)
    return ids


def _none(t, top):
    return torch.full((t, top), -1, dtype=torch.int32)


@pytest.mark.parametrize("t,top,e,kind", [(1, 1, 1, "even"), (1, 8, 64, "even"), (7, 2, 5, "dropped"),
                                          (300, 4, 12, "even"), (513, 8, 60, "dropped"), (1000, 2, 512, "half"),
                                          (2100, 1, 16, "one"), (4000, 8, 256, "even"), (9000, 3, 300, "dropped")])
def test_expert_plan(t, top, e, kind):
    ids = _ids(_gen(t + e), t, top, e, kind)
    plan = pg.expert_plan(ids.cuda(), e)
    counts, offsets, rows, slots = R.lists(ids, e)
    assert plan.counts.tolist() == counts and plan.offsets.tolist() == offsets
    assert plan.rows.tolist() == rows and plan.slots.tolist() == slots


def test_expert_plan_without_tokens_or_experts_rows():
    plan = pg.expert_plan(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 6)
    assert plan.counts.tolist() == [0] * 6 and plan.offsets.tolist() == [0] * 7
    plan = pg.expert_plan(_none(5, 2).cuda(), 6)
    assert plan.offsets.tolist() == [0] * 7 and plan.rows.tolist() == [-1] * 10
    assert plan.slots.tolist() == [[-1, -1]] * 5


def _row_expert(plan_lists, e):
    counts, offsets, rows, _ = plan_lists
    return [(i, offsets[i], offsets[i + 1]) for i in range(e)]


CASES = [(1, 1, 1, 8, 8, "even"), (1, 4, 16, 100, 72, "even"), (3, 2, 6, 64, 130, "dropped"),
         (40, 3, 7, 65, 66, "half"), (130, 2, 5, 136, 200, "dropped"), (400, 4, 9, 257, 120, "even"),
         (300, 2, 4, 96, 520, "one"), (700, 6, 33, 70, 90, "half")]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("t,top,e,n,k,kind", CASES)
def test_expert_linear(dtype, gather, t, top, e, n, k, kind):
    g = _gen(t + n + k)
    ids = _ids(g, t, top, e, kind)
    plan = pg.expert_plan(ids.cuda(), e)
    ls = R.lists(ids, e)
    x = _draw(g, dtype, t if gather else t * top, k)
    w, b = _draw(g, dtype, e, n, k, std=k ** -0.5), _draw(g, dtype, e, n)
    name = R.ACTS[(t + n) % 5]
    y, z = pg.expert_linear(x.cuda(), w.cuda(), plan, b.cuda(), name, gather=gather, preact=True)
    for i, first, end in _row_expert(ls, e):
        src = torch.tensor(ls[2][first:end], dtype=torch.long) // top if gather else torch.arange(first, end)
        want, wz, den = R.linear(x[src], w[i], b[i], name, None)
        R.close(y[first:end], want, den, dtype)
        R.close(z[first:end], wz, den, dtype)
    assert not y[ls[1][-1]:].any() and not z[ls[1][-1]:].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("t,top,e,n,k,kind", CASES)
def test_expert_linear_backward(dtype, gather, t, top, e, n, k, kind):
    g = _gen(t + n + k + 1)
    ids = _ids(g, t, top, e, kind)
    plan = pg.expert_plan(ids.cuda(), e)
    ls = R.lists(ids, e)
    rows = t * top
    x = _draw(g, dtype, t if gather else rows, k)
    w = _draw(g, dtype, e, n, k, std=k ** -0.5)
    dy, z = _draw(g, dtype, rows, n), _draw(g, dtype, rows, n)
    dy[ls[1][-1]:] = math.nan  # rows of no expert are not read
    name = R.ACTS[(t + n + 2) % 5]
    dx, dw, db = pg.expert_linear_backward(dy.cuda(), x.cuda(), w.cuda(), plan, name, z.cuda(), gather=gather)
    wx = torch.zeros(x.shape, dtype=torch.float64)
    dxden = torch.zeros_like(wx)
    wdw = torch.zeros(w.shape, dtype=torch.float64)
    dwden = torch.zeros_like(wdw)
    wdb, dbden = torch.zeros(e, n, dtype=torch.float64), torch.zeros(e, n, dtype=torch.float64)
    for i, first, end in _row_expert(ls, e):
        src = torch.tensor(ls[2][first:end], dtype=torch.long) // top if gather else torch.arange(first, end)
        (a, wdw[i], wdb[i]), (d, dwden[i], dbden[i]) = R.linear_backward(dy[first:end], x[src], w[i], name,
                                                                          z[first:end])
        wx.index_add_(0, src, a)
        dxden.index_add_(0, src, d)
    _check_backward((dx, dw, db), (wx, wdw, wdb), (dxden, dwden, dbden), dtype, name)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_expert_gradients_do_not_mix_experts(dtype):
    """A NaN or infinity in one expert's rows reaches only that expert's gradients, at
    list lengths that end inside every kind of block."""
    t, e, n, k = 260, 6, 72, 136
    g = _gen(2)
    lengths = [1, 63, 0, 65, 130, 1]
    ids = torch.cat([torch.full((c,), i, dtype=torch.int32) for i, c in enumerate(lengths)]).view(t, 1)
    plan = pg.expert_plan(ids.cuda(), e)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, e, n, k)
    dy = _draw(g, dtype, t, n)
    dy[70] = math.nan   # expert 3
    x[255] = math.inf   # expert 4
    dx, dw, db = pg.expert_linear_backward(dy.cuda(), x.cuda(), w.cuda(), plan)
    assert [bool(torch.isfinite(dw[i]).all()) for i in range(e)] == [True, True, True, False, False, True]
    assert [bool(torch.isfinite(db[i]).all()) for i in range(e)] == [True, True, True, False, True, True]
    assert torch.isfinite(dx).all(1).tolist() == [i != 70 for i in range(t)]
    assert not dw[2].any() and not db[2].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_expert_weight_strides(dtype):
    t, top, e, n, k = 50, 2, 3, 40, 56
    g = _gen(6)
    ids = _ids(g, t, top, e, "even")
    plan = pg.expert_plan(ids.cuda(), e)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, e, n, k)
    for pad, rows in ((3, 2), (8, 8)):
        wide = torch.full((e, n + rows, k + pad), math.nan, dtype=dtype, device="cuda")
        wide[:, :n, :k] = w.cuda()
        y = pg.expert_linear(x.cuda(), wide[:, :n, :k], plan, gather=True)
        assert torch.equal(y, pg.expert_linear(x.cuda(), w.cuda(), plan, gather=True))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,top,e,n,kind", [(1, 1, 2, 1, "even"), (5, 3, 8, 70, "dropped"), (200, 8, 16, 1000, "even"),
                                            (33, 2, 4, 2050, "dropped")])
def test_expert_combine(dtype, t, top, e, n, kind):
    g = _gen(t + n)
    ids = _ids(g, t, top, e, kind)
    plan = pg.expert_plan(ids.cuda(), e)
    slots = torch.tensor(R.lists(ids, e)[3]).view(t, top)
    rows, res = _draw(g, dtype, t * top, n), _draw(g, dtype, t, n)
    weights = torch.rand(t, top, generator=g)
    held = (slots >= 0).double()[:, :, None]
    picked = rows.double()[slots.clamp_min(0)] * held
    for wt, r in ((weights, res), (None, None)):
        y = pg.expert_combine(rows.cuda(), plan, None if wt is None else wt.cuda(), None if r is None else r.cuda())
        terms = picked * (1.0 if wt is None else wt.double()[:, :, None])
        want, den = terms.sum(1), terms.abs().sum(1)
        if r is not None:
            want, den = want + r.double(), den + r.double().abs()
        R.close(y, want, den, dtype, slope=1.0)
    # backward: a pair's row gets its weight times its token's gradient
    dy = _draw(g, dtype, t, n)
    drows, dweights = pg.expert_combine_backward(dy.cuda(), rows.cuda(), plan, weights.cuda())
    wrows = torch.zeros(t * top, n, dtype=torch.float64)
    wrows[slots[slots >= 0]] = (weights.double()[:, :, None] * dy.double()[:, None, :])[slots >= 0]
    R.close(drows, wrows, wrows.abs(), dtype, slope=1.0)
    wdw, dden = (picked * dy.double()[:, None, :]).sum(2), (picked * dy.double()[:, None, :]).abs().sum(2)
    R.close(dweights, wdw, dden, torch.float32, slope=1.0)


# ---- streams, graphs, determinism -----------------------------------------------------


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_layers_repeat_bitwise_on_streams_and_in_graphs(dtype):
    t, top, e, n, k = 200, 2, 8, 264, 328
    g = _gen(4)
    x, w = _draw(g, dtype, t, k).cuda(), _draw(g, dtype, e, n, k).cuda()
    ids = _ids(g, t, top, e, "even").cuda()
    logits = _draw(g, dtype, t, e).cuda()

    def work():
        weights, chosen = pg.route(logits, top)
        plan = pg.expert_plan(ids, e)
        h, z = pg.expert_linear(x, w, plan, act="silu", gather=True, preact=True)
        y = pg.expert_combine(h, plan, weights)
        dx, dw, db = pg.expert_linear_backward(h, x, w, plan, "silu", z, gather=True)
        ly, lz = pg.linear(x, w[0], act="gelu", preact=True)
        return [weights, chosen, h, y, dx, dw, db, ly, *pg.linear_backward(ly, x, w[0], "gelu", lz)]

    first = work()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = work()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = work()
    for v in held:
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_result_on_the_stream_that_is_given():
    x, w = torch.randn(300, 256, device="cuda"), torch.randn(200, 256, device="cuda")
    want = pg.linear(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        y = pg.linear(x, w, stream=s)
        s.synchronize()
        assert torch.equal(y, want)


def test_large_offsets():
    """Row offsets beyond 2^31 elements: the last rows of a tall matrix."""
    t, k, n = 2 ** 20 + 3, 2100, 40
    x = torch.empty(t, k, dtype=torch.bfloat16, device="cuda")
    x.fill_(0)
    tail = _draw(_gen(1), torch.bfloat16, 5, k)
    x[-5:] = tail.cuda()
    w = _draw(_gen(2), torch.bfloat16, n, k, std=k ** -0.5)
    y = pg.linear(x, w.cuda())
    want, _, den = R.linear(tail, w, None, "none", None)
    R.close(y[-5:], want, den, torch.bfloat16)
    assert not y[:-5].any()


# ---- limits of float32, empty extents, failure detection --------------------------------


@pytest.mark.parametrize("t", [2, 90])
def test_float32_range(t):
    """Values near the largest float, whose first part would round to infinity, and small
    ones: the three bfloat16 parts keep 24 bits down to about 2^-109 (the last part then
    still is a normal bfloat16 or exact)."""
    n, k = 70, 130
    g = _gen(t)
    x, w = torch.randn(t, k, generator=g), torch.randn(n, k, generator=g)
    big = x.clone()
    big[:, 3] = torch.finfo(torch.float32).max * torch.sign(x[:, 3])
    small = x * 2.0 ** -100
    for a, scale in ((big, 2.0 ** -20), (small, 2.0 ** 20)):
        b = w * scale
        y = pg.linear(a.cuda(), b.cuda())
        want, _, den = R.linear(a, b, None, "none", None)
        R.close(y, want, den, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_gradients_of_empty_extents(dtype):
    def empty(*shape):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    dx, dw, db = pg.linear_backward(empty(7, 0), empty(7, 5), empty(0, 5))
    assert dx.shape == (7, 5) and not dx.any() and dw.shape == (0, 5) and db.shape == (0,)
    dx, dw, db = pg.linear_backward(torch.ones(7, 3, dtype=dtype, device="cuda"), empty(7, 0), empty(3, 0))
    assert dx.shape == (7, 0) and dw.shape == (3, 0) and db.tolist() == [7.0] * 3
    plan = pg.expert_plan(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3)
    w = torch.ones(3, 4, 6, dtype=dtype, device="cuda")
    assert pg.expert_linear(empty(0, 6), w, plan, gather=True).shape == (0, 4)
    dx, dw, db = pg.expert_linear_backward(empty(0, 4), empty(0, 6), w, plan, gather=True)
    assert dx.shape == (0, 6) and not dw.any() and not db.any()
    assert pg.expert_combine(empty(0, 4), plan).shape == (0, 4)
    plan = pg.expert_plan(_none(5, 2).cuda(), 3)  # tokens, but none of them has an expert
    x = torch.ones(5, 6, dtype=dtype, device="cuda")
    y, z = pg.expert_linear(x, w, plan, gather=True, preact=True)
    assert not y.any() and not z.any()
    dx, dw, db = pg.expert_linear_backward(y, x, w, plan, gather=True)
    assert not dx.any() and not dw.any() and not db.any()
    drows, dweights = pg.expert_combine_backward(x, torch.ones(10, 6, dtype=dtype, device="cuda"), plan,
                                                 torch.ones(5, 2, device="cuda"))
    assert not drows.any() and not dweights.any()


@pytest.mark.parametrize("bn,split", [(64, 0), (128, 0), (256, 0), (128, 3), (256, 7)])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_linear_every_tile_width_and_k_slices(dtype, bn, split):
    t, n, k = 400, 600, 1100
    g = _gen(bn + split)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, n, k, std=k ** -0.5)
    b, r = _draw(g, dtype, n), _draw(g, dtype, t, n)
    dy = _draw(g, dtype, t, n)
    pg.force_plan(bn, split)
    try:
        y, z = pg.linear(x.cuda(), w.cuda(), b.cuda(), "gelu", r.cuda(), preact=True)
        again = pg.linear(x.cuda(), w.cuda(), b.cuda(), "gelu", r.cuda())
        grads = pg.linear_backward(dy.cuda(), x.cuda(), w.cuda())
    finally:
        pg.force_plan(0, 0)
    want, wz, den = R.linear(x, w, b, "gelu", r)
    R.close(y, want, den, dtype)
    R.close(z, wz, den, dtype)
    assert torch.equal(y, again)  # slices are added in a fixed order
    want, den = R.linear_backward(dy, x, w, "none", z.cpu())
    _check_backward(grads, want, den, dtype, "none")


def test_half_tiles_of_a_last_wave():
    """More tiles of 256 x 256 than SM pairs by a few: the last wave's run as halves, the
    very last of them past the rows' end."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    t, n, k = 256 * (pairs + 5) - 200, 250, 1024  # one row of tiles; the last tile holds 56 rows
    g = _gen(3)
    x, w = _draw(g, torch.bfloat16, t, k), _draw(g, torch.bfloat16, n, k, std=k ** -0.5)
    pg.force_plan(256, 0)
    try:
        y = pg.linear(x.cuda(), w.cuda())
    finally:
        pg.force_plan(0, 0)
    want, _, den = R.linear(x, w, None, "none", None)
    R.close(y, want, den, torch.bfloat16)


def test_expired_wait_is_reported():
    """A loader that issues nothing (a test hook): the kernel's bounded waits run out, the
    call's status says so, and the next call is right again."""
    x, w = torch.randn(300, 256, device="cuda").bfloat16(), torch.randn(200, 256, device="cuda").bfloat16()
    want = pg.linear(x, w)
    limit = pg.set_wait_timeout(50_000_000)
    flags = pg.debug_flags(pg.SGEMM_DEBUG_STALL_PRODUCER)
    try:
        pg.linear(x, w)
        assert pg.device_status() == pg.SGEMM_ERR_TIMEOUT
    finally:
        pg.debug_flags(flags)
        pg.set_wait_timeout(limit)
    assert torch.equal(pg.linear(x, w), want) and pg.device_status() == 0


def test_injected_host_faults_fail_cleanly():
    x, w = torch.randn(300, 256, device="cuda").bfloat16(), torch.randn(200, 256, device="cuda").bfloat16()
    pg.linear(x, w)
    before = pg.launch_count()
    pg.debug_flags(pg.SGEMM_DEBUG_FAIL_TENSOR_MAP)
    try:
        with pytest.raises(pg.SgemmError) as e:
            pg.linear(x, w)
        assert e.value.code == pg.SGEMM_ERR_TENSOR_MAP
    finally:
        pg.debug_flags(0)
    pg.debug_flags(pg.SGEMM_DEBUG_FAIL_ALLOC)
    s = torch.cuda.Stream()  # without a workspace yet
    try:
        with pytest.raises(pg.SgemmError) as e:
            pg.linear(x.float(), w.float(), stream=s)
        assert e.value.code == pg.SGEMM_ERR_ALLOC
    finally:
        pg.debug_flags(0)
    assert pg.launch_count() == before


def test_given_workspace_is_used_and_its_size_checked():
    x, w = torch.randn(300, 256, device="cuda"), torch.randn(200, 256, device="cuda")
    want = pg.linear(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    try:
        pg.set_workspace(torch.empty(8 << 20, dtype=torch.uint8, device="cuda"), stream=s)
        graph = torch.cuda.CUDAGraph()  # nothing is allocated: the first call can be captured
        with torch.cuda.graph(graph, stream=s):
            y = pg.linear(x, w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        pg.set_workspace(torch.empty(1024, dtype=torch.uint8, device="cuda"), stream=s)
        with pytest.raises(pg.SgemmError) as e:
            pg.linear(x, w, stream=s)
        assert e.value.code == pg.SGEMM_ERR_WORKSPACE
    finally:
        pg.set_workspace(None, stream=s)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_gradients_over_a_workspace_of_nan(dtype):
    """What lies in the workspace before a call (here NaN everywhere) reaches no result, with
    rows long enough to be padded to whole lines."""
    t, n, k, e, top = 150, 530, 1100, 4, 2
    g = _gen(12)
    x, w, dy = _draw(g, dtype, t, k), _draw(g, dtype, e, n, k, std=k ** -0.5), _draw(g, dtype, t * top, n)
    z = _draw(g, dtype, t * top, n)
    ids = _ids(g, t, top, e, "dropped").cuda()
    plan = pg.expert_plan(ids, e)
    xc, wc, dyc, zc = (v.cuda() for v in (x, w, dy, z))
    want, den = R.linear_backward(dy[:t], x, w[0], "gelu", z[:t])
    experts = pg.expert_linear_backward(dyc, xc, wc, plan, "gelu", zc, gather=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    try:
        space = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        for call in (lambda: pg.linear_backward(dyc[:t], xc, wc[0], "gelu", zc[:t], stream=s),
                     lambda: pg.expert_linear_backward(dyc, xc, wc, plan, "gelu", zc, gather=True, stream=s)):
            space.fill_(255)
            torch.cuda.synchronize()
            pg.set_workspace(space, stream=s)
            got = call()
            torch.cuda.synchronize()
            if got[1].dim() == 2:
                _check_backward(got, want, den, dtype, "gelu")
            else:
                assert all(torch.equal(a, b) and bool(torch.isfinite(a).all()) for a, b in zip(got, experts))
    finally:
        pg.set_workspace(None, stream=s)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("pad_x,pad_w", [(0, 0), (1, 0), (0, 3), (5, 1)])
@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 16, 17])
def test_linear_few_rows_of_any_alignment(dtype, t, pad_x, pad_w):
    """Rows long enough for whole steps of a warp's loads and an end, wherever they start."""
    n, k = 70, 2104
    g = _gen(t + 10 * pad_x + pad_w)
    x, w, r = _draw(g, dtype, t, k), _draw(g, dtype, n, k, std=k ** -0.5), _draw(g, dtype, t, n)
    y, z = pg.linear(_strided(x, pad_x, pad_x), _strided(w, pad_w, pad_w), None, "silu", r.cuda(), preact=True)
    want, wz, den = R.linear(x, w, None, "silu", r)
    R.close(y, want, den, dtype)
    R.close(z, wz, den, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,top,e,k", [(2, 4, 16, 2047), (20, 4, 16, 1031), (60, 4, 16, 1031), (40, 4, 8, 1032)])
def test_expert_linear_few_rows_of_any_alignment(dtype, t, top, e, k):
    n = 50
    g = _gen(t + k)
    ids = _ids(g, t, top, e, "dropped")
    ls = R.lists(ids, e)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, e, n, k, std=k ** -0.5)
    y = pg.expert_linear(x.cuda(), w.cuda(), pg.expert_plan(ids.cuda(), e), None, "gelu", gather=True)
    for i, first, end in _row_expert(ls, e):
        src = torch.tensor(ls[2][first:end], dtype=torch.long) // top
        want, _, den = R.linear(x[src], w[i], None, "gelu", None)
        R.close(y[first:end], want, den, dtype)
    assert not y[ls[1][-1]:].any()


def test_linear_few_rows_of_a_large_matrix():
    x, w = _draw(_gen(3), torch.bfloat16, 4, 4096), _draw(_gen(4), torch.bfloat16, 8320, 4096, std=4096 ** -0.5)
    for t in (1, 4):
        want, _, den = R.linear(x[:t], w, None, "none", None)
        R.close(pg.linear(x[:t].cuda(), w.cuda()), want, den, torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("k", [1, 31, 64, 128, 255, 256, 512])
@pytest.mark.parametrize("t", [1, 3, 40])
def test_expert_linear_short_rows(dtype, k, t):
    top, e, n = 2, 12, 40
    g = _gen(t + k)
    ids = _ids(g, t, top, e, "dropped")
    ls = R.lists(ids, e)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, e, n, k, std=k ** -0.5)
    y = pg.expert_linear(x.cuda(), w.cuda(), pg.expert_plan(ids.cuda(), e), None, "silu", gather=True)
    for i, first, end in _row_expert(ls, e):
        src = torch.tensor(ls[2][first:end], dtype=torch.long) // top
        want, _, den = R.linear(x[src], w[i], None, "silu", None)
        R.close(y[first:end], want, den, dtype)
    assert not y[ls[1][-1]:].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k", [(20, 300, 4100), (40, 513, 2050), (300, 257, 1537)])
def test_k_slices_with_every_part_of_the_epilogue(dtype, t, n, k):
    g = _gen(t)
    x, w, b = _draw(g, dtype, t, k), _draw(g, dtype, n, k, std=k ** -0.5), _draw(g, dtype, n)
    r, dy = _draw(g, dtype, t, n), _draw(g, dtype, t, n)
    want, wz, den = R.linear(x, w, b, "gelu", r)
    grads, dens = R.linear_backward(dy, x, w, "silu", wz.to(dtype))
    try:
        for split in (0, 2, 5, 9):
            pg.force_plan(0, split)
            y, z = pg.linear(_strided(x, 3, 1), w.cuda(), b.cuda(), "gelu", _strided(r, 5, 2), preact=True)
            R.close(y, want, den, dtype)
            R.close(z, wz, den, dtype)
            got = pg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), "silu", wz.to(dtype).cuda())
            _check_backward(got, grads, dens, dtype, "silu")
    finally:
        pg.force_plan(0, 0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("split", [0, 3, 8])
def test_k_slices_of_experts(dtype, split):
    """Lists of uneven lengths, some empty, cut along k."""
    t, top, e, n, k = 70, 2, 5, 200, 1100
    g = _gen(21)
    ids = _ids(g, t, top, e, "dropped")
    ls = R.lists(ids, e)
    x, w, b = _draw(g, dtype, t, k), _draw(g, dtype, e, n, k, std=k ** -0.5), _draw(g, dtype, e, n)
    plan = pg.expert_plan(ids.cuda(), e)
    try:
        pg.force_plan(0, split)
        y, z = pg.expert_linear(x.cuda(), w.cuda(), plan, b.cuda(), "relu", gather=True, preact=True)
        dx, _, _ = pg.expert_linear_backward(y, x.cuda(), w.cuda(), plan, gather=True, bias=False, need_dw=False)
    finally:
        pg.force_plan(0, 0)
    wx, xden = torch.zeros(t, k, dtype=torch.float64), torch.zeros(t, k, dtype=torch.float64)
    for i, first, end in _row_expert(ls, e):
        src = torch.tensor(ls[2][first:end], dtype=torch.long) // top
        want, wz, den = R.linear(x[src], w[i], b[i], "relu", None)
        R.close(y[first:end], want, den, dtype)
        R.close(z[first:end], wz, den, dtype)
        got = y[first:end].cpu().double()
        wx.index_add_(0, src, got @ w[i].double())
        xden.index_add_(0, src, got.abs() @ w[i].double().abs())
    R.close(dx, wx, xden, dtype, slope=1.0)
    assert not y[ls[1][-1]:].any() and not z[ls[1][-1]:].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("split", [0, 2, 3, 7])
@pytest.mark.parametrize("gather", [True, False])
def test_k_slices_of_one_experts_gradient(dtype, split, gather):
    """One expert's rows as k of dw, cut into slices of which the last ends inside a block (700 of
    1000 pairs) or is empty, the rows after it NaN."""
    t, n, k, kept = 1000, 72, 136, 700
    g = _gen(31)
    ids = torch.full((t, 1), -1, dtype=torch.int32)
    ids[torch.randperm(t, generator=g)[:kept]] = 0
    plan = pg.expert_plan(ids.cuda(), 1)
    src = torch.nonzero(ids[:, 0] == 0)[:, 0]
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, 1, n, k, std=k ** -0.5)
    dy, z = _draw(g, dtype, t, n), _draw(g, dtype, t, n)
    dy[kept:] = math.nan
    rows = src if gather else torch.arange(kept)
    if not gather:
        x[kept:] = math.nan
    try:
        pg.force_plan(0, split)
        _, dw, db = pg.expert_linear_backward(dy.cuda(), x.cuda(), w.cuda(), plan, "silu", z.cuda(), gather=gather)
    finally:
        pg.force_plan(0, 0)
    want, den = R.linear_backward(dy[:kept], x[rows], w[0], "silu", z[:kept])
    _check_backward((dw[0], db[0]), want[1:], den[1:], dtype, "silu")


# ---- rows without a pair, other empty shapes, long sums ---------------------------------


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("capacity,k", [(2, 1031), (3, 520), (40, 520)])
def test_listed_rows_of_no_pair_read_as_zeros(dtype, capacity, k):
    """Lists of a fixed capacity whose ends name no pair (-1, or a pair past the last), in a plan
    made of four tensors: such a row is act(bias) whichever kernel the sizes lead to, and adds
    nothing to dw."""
    e, n = 6, 72
    t = e * capacity
    g = _gen(capacity + k)
    rows = torch.randperm(t, generator=g).to(torch.int32).view(e, capacity)
    rows[:, capacity - 1] = -1
    rows[2, capacity - 1] = t + 5
    rows[4] = -1
    rows = rows.reshape(-1)
    slots = torch.full((t, 1), -1, dtype=torch.int32)
    held = (rows >= 0) & (rows < t)
    at = torch.nonzero(held)[:, 0]
    slots[rows[held].long(), 0] = at.to(torch.int32)
    plan = pg.ExpertPlan(torch.full((e,), capacity, dtype=torch.int32, device="cuda"),
                         torch.arange(0, t + 1, capacity, dtype=torch.int32, device="cuda"), rows.cuda(), slots.cuda())
    x, w, b = _draw(g, dtype, t, k), _draw(g, dtype, e, n, k, std=k ** -0.5), _draw(g, dtype, e, n)
    dy, z = _draw(g, dtype, t, n), _draw(g, dtype, t, n)
    read = torch.where(held[:, None], x[rows.clamp(0, t - 1).long()], torch.zeros((), dtype=dtype))
    y = pg.expert_linear(x.cuda(), w.cuda(), plan, b.cuda(), "silu", gather=True)
    _, dw, _ = pg.expert_linear_backward(dy.cuda(), x.cuda(), w.cuda(), plan, "silu", z.cuda(), gather=True)
    for i in range(e):
        part = slice(i * capacity, (i + 1) * capacity)
        want, _, den = R.linear(read[part], w[i], b[i], "silu", None)
        R.close(y[part], want, den, dtype)
        (_, want, _), (_, den, _) = R.linear_backward(dy[part], read[part], w[i], "silu", z[part])
        R.close(dw[i], want, den, dtype, slope=1.0, inner=_inner(dtype, "silu"))
    # whatever token 0 holds, a row of no pair does not see it
    x[0] = math.nan
    again = pg.expert_linear(x.cuda(), w.cuda(), plan, b.cuda(), "silu", gather=True)
    sees = (rows == 0).cuda()
    assert torch.isnan(again[sees]).all() and torch.equal(again[~sees], y[~sees])


def _half_spacing(v):
    """Half the distance of bfloat16 values around v (8 significant bits)."""
    return torch.exp2(torch.floor(torch.log2(v.abs())) - 8)


# The tensor core truncates its FP32 sums: an error of at most 2^-23 of the running sum for each
# addition of 16 k, all one way.  A run of additions is kept to 16384 k for bfloat16, so the
# errors of 1024 of them, 2^-13 of the sum of the terms' magnitudes, bound what is lost; the runs
# are added rounded to nearest (2^-18 for 64 of them).
LONG = 2.0 ** -13 + 2.0 ** -18


def test_bfloat16_gradient_over_a_million_rows_of_one_sign():
    t, n, k, e = 2 ** 20 + 37, 72, 136, 2
    ids = torch.zeros(t, 1, dtype=torch.int32, device="cuda")
    plan = pg.expert_plan(ids, e)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.rand(t, k, generator=g, device="cuda").bfloat16()
    dy = torch.rand(t, n, generator=g, device="cuda").bfloat16()
    w = torch.zeros(e, n, k, dtype=torch.bfloat16, device="cuda")
    for gather in (True, False):
        _, dw, _ = pg.expert_linear_backward(dy, x, w, plan, gather=gather, bias=False, need_dx=False)
        want = dy.double().t() @ x.double()
        assert ((dw[0].double() - want).abs() <= _half_spacing(want) + LONG * want).all()
        assert not dw[1].any()


@pytest.mark.parametrize("t", [40, 300])
def test_bfloat16_sums_of_one_sign_over_a_long_k(t):
    """Forward products whose k is no multiple of a run, in one slice and in several."""
    n, k = 200, 5 * 16384 + 1000
    g = torch.Generator(device="cuda").manual_seed(t)
    x = torch.rand(t, k, generator=g, device="cuda").bfloat16()
    w = torch.rand(n, k, generator=g, device="cuda").bfloat16()
    b = torch.rand(n, generator=g, device="cuda").bfloat16()
    want = x.double() @ w.double().t() + b.double()
    try:
        for bn in (64, 128, 256):
            for split in (1, 3):
                pg.force_plan(bn, split)
                y = pg.linear(x, w, b)
                assert ((y.double() - want).abs() <= _half_spacing(want) + LONG * want).all(), (bn, split)
    finally:
        pg.force_plan(0, 0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("n,k", [(9, 0), (0, 5), (0, 0)])
def test_leading_dimensions_over_empty_rows(dtype, n, k):
    x = torch.ones(2, 3, k, dtype=dtype, device="cuda")
    w = torch.ones(n, k, dtype=dtype, device="cuda")
    b = torch.arange(n, device="cuda").to(dtype)
    y, z = pg.linear(x, w, b, residual=torch.ones(2, 3, n, dtype=dtype, device="cuda"), preact=True)
    assert y.shape == z.shape == (2, 3, n)
    assert torch.equal(z, b.expand(2, 3, n)) and torch.equal(y, z + 1)
    dx, dw, db = pg.linear_backward(torch.ones(2, 3, n, dtype=dtype, device="cuda"), x, w, "silu", z)
    assert dx.shape == (2, 3, k) and dw.shape == (n, k) and db.shape == (n,) and not dx.any()


@pytest.mark.parametrize("t", [1, 200])
def test_float32_silu_where_its_logistic_is_below_the_normal_floats(t):
    """From z of -87.3 on, 1 / (1 + exp(-z)) is subnormal (absolute error 2^-150, which z makes
    at most 2^-143) while z times it is not yet: exp is good to 2^-22, the products to 2^-24."""
    n = 64
    z = torch.linspace(-88.5, -80, n)
    y = pg.linear(torch.zeros(t, 8, device="cuda"), torch.zeros(n, 8, device="cuda"), z.cuda(), "silu")
    want = (z.double() / (1 + torch.exp(-z.double()))).expand(t, n)
    assert ((y.double().cpu() - want).abs() <= 2.0 ** -21 * want.abs() + 2.0 ** -142).all()
    # its derivative, the slope of a gradient of ones
    dz = torch.exp(z.double()) * (1 + z.double())
    _, _, db = pg.linear_backward(torch.ones(1, n, device="cuda"), torch.zeros(1, 8, device="cuda"),
                                  torch.zeros(n, 8, device="cuda"), "silu", z[None].cuda())
    assert ((db.double().cpu() - dz).abs() <= 2.0 ** -20 * dz.abs() + 2.0 ** -142).all()


@pytest.mark.parametrize("t", [4, 40, 300])
def test_float32_accuracy_on_values_of_one_sign(t):
    """The stated error in the 2-norm at k = 4096, where errors that all point one way add up."""
    n, k = 512, 4096
    g = _gen(t)
    x, w = torch.rand(t, k, generator=g), torch.rand(n, k, generator=g)
    y = pg.linear(x.cuda(), w.cuda()).double().cpu()
    want = x.double() @ w.double().t()
    assert float((y - want).norm() / want.norm()) < 1e-6
