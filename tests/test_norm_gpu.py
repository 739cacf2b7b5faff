"""Layer norm, forward and backward, against its definition in 64 bits: rows from one
element to more than the registers hold, odd lengths, strided and unaligned rows, one
row and many, constant rows, means far from zero, infinities and NaN, both types."""
import math

import pytest
import torch

import precision_gemm_gb300 as pg
from tests._layers_ref import HALF

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
IDS = {torch.float32: "f32", torch.bfloat16: "bf16"}

# Every sum is FP32 in chains and trees of at most 150 additions of its terms, each off by half a
# step, 2^-24; what follows a sum adds a few more roundings of the same terms' sizes.
UNITS = 168 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _release():
    """Streams come back from torch's pool of 32: they leave here without workspaces."""
    yield
    pg.workspace_release()


@pytest.fixture(autouse=True)
def _healthy():
    pg.load_library()
    pg.device_status()
    yield
    assert pg.device_status() == 0


def _draw(g, dtype, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _strided(x, pad, offset=0):
    """A CUDA copy of x whose rows are pad elements apart more than they are long, `offset`
    elements into the storage; the gaps hold NaN."""
    r, c = x.shape
    buf = torch.full((offset + r * (c + pad),), math.nan, dtype=x.dtype, device="cuda")
    view = buf[offset:].view(r, c + pad)[:, :c]
    view.copy_(x)
    return view


def forward(x, w, b, eps):
    """(y, mean, rstd) and the sizes that their errors go by."""
    x = x.double()
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(n, dtype=torch.float64) if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    h = (x - mean) * rstd
    size = x.abs().mean(1, keepdim=True)
    return ((h * w + b, mean[:, 0], rstd[:, 0]),
            (w.abs() * (rstd * size + h.abs()) + b.abs(), size[:, 0], rstd[:, 0]))


def backward(dy, x, w, mean, rstd, r):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    g = dy if w is None else dy * w.double()
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = rstd * (g - c1 - h * c2)
    den = rstd * (g.abs() + g.abs().mean(1, keepdim=True) + h.abs() * (g * h).abs().mean(1, keepdim=True))
    if r is not None:
        dx, den = dx + r.double(), den + r.double().abs()
    return (dx, (dy * h).sum(0), dy.sum(0)), (den, (dy * h).abs().sum(0), dy.abs().sum(0))


def close(got, want, den, dtype):
    got = got.double().cpu()
    assert got.shape == want.shape
    exact = UNITS * den
    tol = exact + (HALF * (want.abs() + exact) if dtype == torch.bfloat16 else 0.0)
    err = (got - want).abs()
    assert (err <= tol + 1e-40).all(), float((err / (tol + 1e-40)).max())


def _check(g, dtype, t, n, shift=0.0, eps=1e-5):
    x = _draw(g, dtype, t, n) + shift
    w, b, dy, r = (_draw(g, dtype, *s) for s in ((n,), (n,), (t, n), (t, n)))
    y, mean, rstd = pg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps, stats=True)
    want, den = forward(x, w, b, eps)
    for a, v, d, ty in zip((y, mean, rstd), want, den, (dtype, torch.float32, torch.float32)):
        close(a, v, d, ty)
    got = pg.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd, r.cuda())
    want, den = backward(dy, x, w, mean.cpu(), rstd.cpu(), r)
    for a, v, d in zip(got, want, den):
        close(a, v, d, dtype)


SIZES = [(1, 2), (1, 4096), (2, 8), (3, 5), (4, 64), (5, 255), (7, 256), (33, 257), (1000, 48), (700, 777), (9, 2047),
         (40, 2048), (129, 2056), (3, 4097), (640, 4096), (2, 8192), (50, 8200), (9, 16384), (5, 16385), (3, 32768),
         (2, 33000), (300, 32800)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n", SIZES)
def test_norm(dtype, t, n):
    _check(torch.Generator().manual_seed(t * 31 + n), dtype, t, n)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n", [(20000, 64), (9000, 1030), (5000, 4096)])
def test_norm_many_rows(dtype, t, n):
    _check(torch.Generator().manual_seed(n), dtype, t, n)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t", [1, 3, 33, 4099])
@pytest.mark.parametrize("n", [2, 9, 63, 64, 65, 100, 128, 129])
def test_norm_narrow_rows(dtype, t, n):
    """Rows that a part of a warp holds, several of them to a warp, whose last ones may be missing."""
    _check(torch.Generator().manual_seed(t + n), dtype, t, n)


@pytest.mark.parametrize("n", [100, 4096, 9000])
def test_norm_mean_far_from_zero(n):
    """A mean a thousand times the spread: the squares are taken around it."""
    _check(torch.Generator().manual_seed(n), torch.float32, 30, n, shift=1000.0)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_norm_constant_rows_and_rows_of_one(dtype):
    x = torch.full((3, 320), 3.25, dtype=dtype, device="cuda")
    y, mean, rstd = pg.layer_norm(x, eps=1e-3, stats=True)
    assert not y.any() and (mean == 3.25).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-3 ** -0.5), rtol=1e-6)
    b = torch.tensor([0.5], dtype=dtype, device="cuda")
    y, mean, rstd = pg.layer_norm(x[:, :1], b, b, stats=True)  # one element: always its own mean
    assert (y == 0.5).all()
    dx, dw, db = pg.layer_norm_backward(torch.ones_like(y), x[:, :1], b, mean, rstd)
    assert not dx.any() and not dw.any() and db.tolist() == [3.0]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,pad,offset", [(7, 96, 3, 1), (90, 1000, 8, 8), (90, 1000, 5, 0), (33, 8192, 8, 3),
                                            (20, 33000, 1, 1), (1, 264, 9, 0)])
def test_norm_strides_and_alignment(dtype, t, n, pad, offset):
    g = torch.Generator().manual_seed(n + pad)
    x, w, b, dy, r = (_draw(g, dtype, *s) for s in ((t, n), (n,), (n,), (t, n), (t, n)))
    out = _strided(torch.zeros(t, n, dtype=dtype), pad, offset)
    xs = _strided(x, pad, offset)
    got, mean, rstd = pg.layer_norm(xs, w.cuda(), b.cuda(), stats=True, out=out)
    assert got is out
    want, den = forward(x, w, b, 1e-5)
    close(out, want[0], den[0], dtype)
    gaps = out.as_strided((t, pad), (n + pad, 1), out.storage_offset() + n)[:t - 1]
    assert torch.isnan(gaps).all()
    grads = pg.layer_norm_backward(_strided(dy, pad, offset), xs, w.cuda(), mean, rstd, _strided(r, pad, offset))
    want, den = backward(dy, x, w, mean.cpu(), rstd.cpu(), r)
    for a, v, d in zip(grads, want, den):
        close(a, v, d, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("n", [72, 9001])
def test_norm_without_weight_or_bias_and_skipped_gradients(dtype, n):
    g = torch.Generator().manual_seed(4)
    t = 70
    x, w, b, dy, r = (_draw(g, dtype, *s) for s in ((t, n), (n,), (n,), (t, n), (t, n)))
    cx, cw, cdy = x.cuda(), w.cuda(), dy.cuda()
    for ww, bb in ((None, None), (w, None), (None, b)):
        y, mean, rstd = pg.layer_norm(cx, None if ww is None else cw, None if bb is None else b.cuda(), stats=True)
        want, den = forward(x, ww, bb, 1e-5)
        close(y, want[0], den[0], dtype)
        assert torch.equal(y, pg.layer_norm(cx, None if ww is None else cw, None if bb is None else b.cuda()))
        dx, dw, db = pg.layer_norm_backward(cdy, cx, None if ww is None else cw, mean, rstd)
        want, den = backward(dy, x, ww, mean.cpu(), rstd.cpu(), None)
        close(dx, want[0], den[0], dtype)
        close(db, want[2], den[2], dtype)
        if ww is None:
            assert dw is None
        else:
            close(dw, want[1], den[1], dtype)
    whole = pg.layer_norm_backward(cdy, cx, cw, mean, rstd, r.cuda())
    dx, dw, db = pg.layer_norm_backward(cdy, cx, cw, mean, rstd, r.cuda(), bias=False, need_dw=False)
    assert dw is None and db is None and torch.equal(dx, whole[0])
    dx, dw, db = pg.layer_norm_backward(cdy, cx, cw, mean, rstd, need_dx=False)
    assert dx is None and torch.equal(dw, whole[1]) and torch.equal(db, whole[2])


def test_norm_leading_dimensions_and_no_rows():
    g = torch.Generator().manual_seed(5)
    x, w = _draw(g, torch.float32, 2, 3, 40).cuda(), _draw(g, torch.float32, 40).cuda()
    y, mean, rstd = pg.layer_norm(x, w, stats=True)
    assert y.shape == x.shape and mean.shape == rstd.shape == (2, 3)
    flat = pg.layer_norm(x.view(6, 40), w)
    assert torch.equal(y.view(6, 40), flat)
    dx, dw, db = pg.layer_norm_backward(y, x, w, mean, rstd)
    assert dx.shape == x.shape
    empty = torch.empty(0, 40, device="cuda")
    y, mean, rstd = pg.layer_norm(empty, w, stats=True)
    assert y.shape == (0, 40) and mean.shape == (0,)
    dx, dw, db = pg.layer_norm_backward(empty, empty, w, mean, rstd)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("n", [64, 3000, 33000])
def test_norm_infinities_and_nan_stay_in_their_rows(dtype, n):
    g = torch.Generator().manual_seed(6)
    x = _draw(g, dtype, 9, n)
    x[2, 5], x[7, n - 1] = math.inf, math.nan
    y = pg.layer_norm(x.cuda()).cpu()
    assert torch.isnan(y).all(1).tolist() == [i in (2, 7) for i in range(9)]
    assert torch.isfinite(y[[0, 1, 3, 4, 5, 6, 8]]).all()


@pytest.mark.parametrize("n", [40, 3000])
def test_norm_backward_against_differences(n):
    """Differences of the 64-bit norm around the point, step 1e-5: their own error is of order
    1e-10, the FP32 gradient's 1e-6 of its terms."""
    t = 12
    g = torch.Generator().manual_seed(n)
    x, w, b, dy = (torch.randn(*s, generator=g) for s in ((t, n), (n,), (n,), (t, n)))
    y, mean, rstd = pg.layer_norm(x.cuda(), w.cuda(), b.cuda(), stats=True)
    grads = pg.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)

    def loss(x, w, b):
        return float((forward(x, w, b, 1e-5)[0][0] * dy.double()).sum())

    h = 1e-5
    for i, (v, grad) in enumerate(zip((x, w, b), grads)):
        u = torch.randn(v.shape, generator=g, dtype=torch.float64)
        at = [x.double(), w.double(), b.double()]
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * u, at[i] - h * u
        diff = (loss(*up) - loss(*down)) / (2 * h)
        grad = grad.double().cpu()
        assert abs(diff - float((grad * u).sum())) <= 2e-5 * float((grad.abs() * u.abs()).sum()), i


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_norm_repeats_bitwise_on_streams_and_in_graphs(dtype):
    g = torch.Generator().manual_seed(8)
    sets = [[_draw(g, dtype, *s).cuda() for s in ((t, n), (n,), (n,), (t, n))] for t, n in ((700, 1000), (90, 9000))]

    def work():
        out = []
        for x, w, b, dy in sets:
            y, mean, rstd = pg.layer_norm(x, w, b, stats=True)
            out += [y, mean, rstd, *pg.layer_norm_backward(dy, x, w, mean, rstd, residual=y)]
        return out

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
    x, w, b, _ = sets[0]
    y = pg.layer_norm(x, w, b, stream=s)
    s.synchronize()
    assert torch.equal(y, first[0])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n", [(5, 64), (300, 777), (700, 4096), (9, 16384), (4, 16386)])
def test_norm_in_place(dtype, t, n):
    """y over x, and dx over the gradient that is added to it."""
    g = torch.Generator().manual_seed(n)
    x, dy, r = (_draw(g, dtype, t, n).cuda() for _ in range(3))
    w = _draw(g, dtype, n).cuda()
    want, mean, rstd = pg.layer_norm(x, w, w, stats=True)
    dx = pg.layer_norm_backward(dy, x, w, mean, rstd, r)[0]
    lib, code = pg.load_library(), 0 if dtype == torch.float32 else 1
    rc = lib.sgemm_layer_norm_backward(code, t, n, dy.data_ptr(), n, x.data_ptr(), n, w.data_ptr(), mean.data_ptr(),
                                       rstd.data_ptr(), r.data_ptr(), n, r.data_ptr(), n, None, None,
                                       torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(r, dx)
    y = x.clone()
    assert pg.layer_norm(y, w, w, out=y) is y and torch.equal(y, want)


def test_norm_large_offsets():
    """Rows that start beyond 2^31 elements, the last ones of a tall matrix."""
    t, n = 2 ** 20 + 3, 2100
    x = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    tail = _draw(torch.Generator().manual_seed(1), torch.bfloat16, 5, n)
    x[-5:] = tail.cuda()
    y, mean, rstd = pg.layer_norm(x, stats=True)
    want, den = forward(tail, None, None, 1e-5)
    close(y[-5:], want[0], den[0], torch.bfloat16)
    assert not y[:-5].any()
    dx, _, db = pg.layer_norm_backward(x, x, None, mean, rstd)
    want, den = backward(tail, tail, None, mean[-5:].cpu(), rstd[-5:].cpu(), None)
    close(dx[-5:], want[0], den[0], torch.bfloat16)
    close(db, want[2], den[2], torch.bfloat16)
    assert not dx[:-5].any()


def test_norm_binding_refuses_mismatched_tensors():
    x = torch.randn(6, 16, device="cuda")
    w = torch.randn(16, device="cuda")
    y, mean, rstd = pg.layer_norm(x, w, stats=True)
    before = pg.launch_count()
    bad = [lambda: pg.layer_norm(x, w[:8]), lambda: pg.layer_norm(x, w.double()), lambda: pg.layer_norm(x.half(), w),
           lambda: pg.layer_norm(x, w, w.cpu()), lambda: pg.layer_norm(x.t(), x[:, 0]),
           lambda: pg.layer_norm(x, w, out=x[:3]), lambda: pg.layer_norm(x, x[:, :1].expand(6, 16)[0][::2]),
           lambda: pg.layer_norm_backward(y[:5], x, w, mean, rstd),
           lambda: pg.layer_norm_backward(y, x, w, mean[:5], rstd),
           lambda: pg.layer_norm_backward(y, x, w, mean, rstd.double()),
           lambda: pg.layer_norm_backward(y, x, w, mean, rstd, residual=y[:, :8])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for eps in (-1.0, math.nan, math.inf):
        with pytest.raises(pg.SgemmError):
            pg.layer_norm(x, w, eps=eps)
    with pytest.raises(pg.SgemmError):
        pg.layer_norm(x[:, :0])
    assert pg.launch_count() == before


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("n", [3, 64, 100, 777, 1000, 4095, 7168, 9001, 16384, 20000, 32769])
def test_norm_equal_values_are_their_mean(dtype, n):
    """Rows of one value each: it is their mean to the bit, and every h is zero, whatever 1 / n and the
    sums round to (the values' differences from any float near them are few of its last places, whose
    sums are exact)."""
    x = torch.tensor([3.25, 1000.0, 100.1, -777.7, 7.0, 12345.6]).to(dtype)[:, None].expand(6, n).contiguous().cuda()
    b = _draw(torch.Generator().manual_seed(n), dtype, n).cuda()
    y, mean, rstd = pg.layer_norm(x, stats=True)
    assert not y.any() and torch.equal(mean, x[:, 0].float())
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    assert torch.equal(pg.layer_norm(x, None, b), b.expand(6, n))
    near = torch.full((9, n), 2.0 ** -10, dtype=dtype, device="cuda")  # a mean within h's unit, beside others
    near[4] = 1000
    assert torch.equal(pg.layer_norm(near)[3], pg.layer_norm(near[:4])[3])


@pytest.mark.parametrize("dtype,shift", [(torch.float32, 1e3), (torch.float32, -1e5), (torch.bfloat16, 100.0)])
@pytest.mark.parametrize("t,n", [(40, 100), (3, 1000), (30, 4096), (9, 7169), (6, 16384), (4, 20000), (3, 32771)])
def test_norm_mean_far_from_zero_costs_no_bits(dtype, shift, t, n):
    """The values' differences from a float near their mean are exact, so h is off by the sums of such
    differences alone: UNITS of their mean magnitude, which is at most 1 / rstd, and UNITS of h for
    rstd; the mean that is returned is rounded once more."""
    g = torch.Generator().manual_seed(n)
    x = (torch.randn(t, n, generator=g) + shift).to(dtype)
    y, mean, rstd = pg.layer_norm(x.cuda(), eps=1e-6, stats=True)
    (want, m, r), _ = forward(x, None, None, 1e-6)
    close(y, want, 1 + 2 * want.abs(), dtype)
    assert ((mean.double().cpu() - m).abs() <= 2.0 ** -24 * m.abs() + UNITS / r).all()
    assert ((rstd.double().cpu() - r).abs() <= UNITS * r).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n", [(5, 64), (300, 777), (700, 4096), (130, 16384), (140, 16386), (300, 32768)])
def test_norm_backward_in_place(dtype, t, n):
    """dx over x, over dy and over the gradient that is added to it: the three gradients are what they are apart."""
    g = torch.Generator().manual_seed(n)
    x, dy, r = (_draw(g, dtype, t, n).cuda() for _ in range(3))
    w = _draw(g, dtype, n).cuda()
    _, mean, rstd = pg.layer_norm(x, w, stats=True)
    want = pg.layer_norm_backward(dy, x, w, mean, rstd, r)
    lib, code = pg.load_library(), 0 if dtype == torch.float32 else 1
    for over in range(3):
        at = [v.clone() for v in (x, dy, r)]
        dw, db = torch.empty_like(w), torch.empty_like(w)
        rc = lib.sgemm_layer_norm_backward(code, t, n, at[1].data_ptr(), n, at[0].data_ptr(), n, w.data_ptr(),
                                           mean.data_ptr(), rstd.data_ptr(), at[2].data_ptr(), n, at[over].data_ptr(), n,
                                           dw.data_ptr(), db.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and all(torch.equal(a, b) for a, b in zip((at[over], dw, db), want)), over


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("n", [64, 777, 4096, 20000])
def test_norm_sums_beyond_float32(dtype, n):
    """Rows of large values beside ordinary ones: a sum beyond the range makes its row NaN, squares beyond
    it make rstd 0 and the row its bias."""
    g = torch.Generator().manual_seed(n)
    x, b = _draw(g, dtype, 6, n), _draw(g, dtype, n).cuda()
    want = pg.layer_norm(x.cuda(), None, b)
    x[1], x[4] = 3e38, x[4] * 1e30
    y, mean, rstd = pg.layer_norm(x.cuda(), None, b, stats=True)
    assert torch.isnan(y[1]).all() and rstd[4] == 0 and torch.equal(y[4], b)
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], want[keep])
