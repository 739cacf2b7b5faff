"""The gated linear layer, forward and backward, against its definition in 64 bits: one
row to several tiles, odd extents, strided and unaligned rows, every activation, forced
tile widths and K slices, both types."""
import math

import pytest
import torch

import precision_gemm_gb300 as pg
from tests import _layers_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
IDS = {torch.float32: "f32", torch.bfloat16: "bf16"}


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


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _draw(g, dtype, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _strided(x, pad, offset=0):
    r, c = x.shape
    buf = torch.full((offset + r * (c + pad),), math.nan, dtype=x.dtype, device="cuda")
    view = buf[offset:].view(r, c + pad)[:, :c]
    view.copy_(x)
    return view


def forward(x, w, bias, name):
    """y, z and their bounds before rounding: a product's terms are summed to 1e-5 of their
    magnitudes' sum, an activation passes that on with a factor of at most 1.13 (R.SLOPE), the
    product of two inexact factors has both errors, and a few roundings follow."""
    _, z, den = R.linear(x, w, bias, "none", None)
    n = z.shape[1] // 2
    g, v = z[:, :n], z[:, n:]
    eg, ev = R.SLOPE * R.NORM * den[:, :n], R.NORM * den[:, n:]
    a = R.act(g, name)
    y = a * v
    return y, z, eg * v.abs() + a.abs() * ev + eg * ev + 2.0 ** -21 * y.abs(), R.NORM * den


def close(got, want, bound, dtype):
    got, want, bound = got.double().cpu(), want.cpu(), bound.cpu()
    assert got.shape == want.shape
    tol = bound + (R.HALF * (want.abs() + bound) if dtype == torch.bfloat16 else 0.0)
    err = (got - want).abs()
    assert (err <= tol + 1e-30).all(), float((err / (tol + 1e-30)).max())


def backward(dy, x, w, name, z):
    """dx, dw, dbias and their terms' magnitudes; values and derivatives of an activation near
    zero are formed from values near 1 (g), which an eighth in the magnitudes covers."""
    n = z.shape[1] // 2
    g, v, dy = z[:, :n].double(), z[:, n:].double(), dy.double()
    a, slope = R.act(g, name), R.dact(g, name)
    extra = 0.0 if name in ("none", "relu") else 0.125
    dz = torch.cat([dy * v * slope, dy * a], 1)
    m = torch.cat([(dy * v).abs() * (slope.abs() + extra), dy.abs() * (a.abs() + extra * g.abs())], 1)
    x, w = x.double(), w.double()
    return (dz @ w, dz.t() @ x, dz.sum(0)), (m @ w.abs(), m.t() @ x.abs(), m.sum(0))


def _check_backward(got, want, den, dtype):
    inner = R.HALF if dtype == torch.bfloat16 else 0.0  # dz is rounded before the products
    for i, (a, b, d) in enumerate(zip(got, want, den)):
        R.close(a, b, d, dtype, slope=1.0, inner=inner if i < 2 else 0.0)


SIZES = [(1, 1, 1), (1, 130, 3), (1, 2048, 520), (2, 4096, 512), (3, 64, 64), (4, 33, 777), (5, 1000, 777),
         (8, 96, 2048), (16, 257, 130), (17, 257, 129), (33, 640, 256), (64, 128, 64), (130, 300, 777),
         (257, 513, 1000), (300, 256, 65), (1500, 300, 777)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k", SIZES)
def test_gated_linear(dtype, t, n, k):
    g = _gen(t * 7 + n * 3 + k)
    x, w, b = _draw(g, dtype, t, k), _draw(g, dtype, 2 * n, k, std=k ** -0.5), _draw(g, dtype, 2 * n)
    name = R.ACTS[(t + n + k) % 5]
    y, z = pg.gated_linear(x.cuda(), w.cuda(), b.cuda(), name, preact=True)
    want, wz, bound, zb = forward(x, w, b, name)
    close(y, want, bound, dtype)
    close(z, wz, zb, dtype)
    assert torch.equal(y, pg.gated_linear(x.cuda(), w.cuda(), b.cuda(), name))
    y = pg.gated_linear(x.cuda(), w.cuda())
    want, _, bound, _ = forward(x, w, None, "silu")
    close(y, want, bound, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("t", [2, 200])
def test_gated_activations_over_their_range(dtype, name, t):
    n, k = 192, 32
    g = _gen(5)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, 2 * n, k, std=k ** -0.5)
    b = torch.cat([torch.linspace(-12, 12, n), torch.linspace(3, -3, n)]).to(dtype)
    x[0] = 0
    y = pg.gated_linear(x.cuda(), w.cuda(), b.cuda(), name)
    want, _, bound, _ = forward(x, w, b, name)
    close(y, want, bound, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k,pad,offset", [(2, 70, 100, 3, 1), (6, 70, 100, 3, 1), (140, 200, 136, 5, 3),
                                              (140, 200, 136, 8, 8), (300, 130, 64, 1, 0), (1, 64, 72, 7, 2)])
def test_gated_strides_and_alignment(dtype, t, n, k, pad, offset):
    g = _gen(t + pad)
    x, w, b = _draw(g, dtype, t, k), _draw(g, dtype, 2 * n, k, std=k ** -0.5), _draw(g, dtype, 2 * n)
    out = _strided(torch.zeros(t, n, dtype=dtype), pad, offset)
    z = _strided(torch.zeros(t, 2 * n, dtype=dtype), pad, offset)
    xs, ws = _strided(x, pad, offset), _strided(w, pad, offset)
    got = pg.gated_linear(xs, ws, b.cuda(), "gelu", out=out, preact=z)
    assert got is out
    want, wz, bound, zb = forward(x, w, b, "gelu")
    close(out, want, bound, dtype)
    close(z, wz, zb, dtype)
    for v, cols in ((out, n), (z, 2 * n)):
        gaps = v.as_strided((t, pad), (cols + pad, 1), offset + cols)[:t - 1]
        assert torch.isnan(gaps).all()
    dy = _draw(g, dtype, t, n)
    grads = pg.gated_linear_backward(_strided(dy, pad, offset), xs, ws, z, "gelu")
    want, den = backward(dy, x, w, "gelu", z.cpu())
    _check_backward(grads, want, den, dtype)
    dx, dw, db = pg.gated_linear_backward(_strided(dy, pad, offset), xs, ws, z, "gelu", need_dw=False, bias=False)
    assert dw is None and db is None and torch.equal(dx, grads[0])
    dx, dw, db = pg.gated_linear_backward(_strided(dy, pad, offset), xs, ws, z, "gelu", need_dx=False)
    assert dx is None and torch.equal(dw, grads[1]) and torch.equal(db, grads[2])
    dx, dw, db = pg.gated_linear_backward(_strided(dy, pad, offset), xs, ws, z, "gelu", need_dx=False, need_dw=False)
    assert dx is None and dw is None and torch.equal(db, grads[2])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 70, 130), (5, 64, 64), (63, 65, 66), (130, 300, 77), (257, 130, 200),
                                   (640, 256, 384), (1300, 100, 150)])
def test_gated_linear_backward(dtype, t, n, k):
    g = _gen(t + n + k)
    name = R.ACTS[(t + n + k) % 5]
    x, w, dy = _draw(g, dtype, t, k), _draw(g, dtype, 2 * n, k, std=k ** -0.5), _draw(g, dtype, t, n)
    z = _draw(g, dtype, t, 2 * n, std=2.0)
    got = pg.gated_linear_backward(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), name)
    want, den = backward(dy, x, w, name, z)
    _check_backward(got, want, den, dtype)


@pytest.mark.parametrize("name", R.ACTS)
def test_gated_backward_against_differences(name):
    """Directional differences of the 64-bit layer around the point, step 1e-5: their own
    error is of order 1e-10, the FP32 gradient's 1e-6 of the terms' sizes."""
    t, n, k = 40, 50, 60
    g = _gen(11)
    x, w, b = (torch.randn(*s, generator=g) for s in ((t, k), (2 * n, k), (2 * n,)))
    w = w * k ** -0.5
    dy = torch.randn(t, n, generator=g)
    z64 = x.double() @ w.double().t() + b.double()
    # relu has no derivative at zero: no pre-activation within a step of it
    assert name != "relu" or float(z64[:, :n].abs().min()) > 1e-4
    y, z = pg.gated_linear(x.cuda(), w.cuda(), b.cuda(), name, preact=True)
    grads = pg.gated_linear_backward(dy.cuda(), x.cuda(), w.cuda(), z, name)

    def loss(x, w, b):
        z = x @ w.t() + b
        return float((R.act(z[:, :n], name) * z[:, n:] * dy.double()).sum())

    h = 1e-5
    for i, (v, grad) in enumerate(zip((x, w, b), grads)):
        u = torch.randn(v.shape, generator=g, dtype=torch.float64)
        at = [x.double(), w.double(), b.double()]
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * u, at[i] - h * u
        diff = (loss(*up) - loss(*down)) / (2 * h)
        grad = grad.double().cpu()
        assert abs(diff - float((grad * u).sum())) <= 2e-5 * float((grad.abs() * u.abs()).sum()), (name, i)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_gated_empty_extents_and_leading_dimensions(dtype):
    def empty(*shape):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    g = _gen(1)
    b = _draw(g, dtype, 18)
    y, z = pg.gated_linear(empty(4, 0), empty(18, 0), b.cuda(), "silu", preact=True)
    want, wz, bound, zb = forward(torch.zeros(4, 0), torch.zeros(18, 0), b, "silu")
    close(y, want, bound, dtype)
    close(z, wz, zb, dtype)
    assert pg.gated_linear(empty(0, 5), empty(18, 5)).shape == (0, 9)
    assert pg.gated_linear(empty(3, 5), empty(0, 5)).shape == (3, 0)
    x, w = _draw(g, dtype, 2, 3, 40), _draw(g, dtype, 48, 40)
    y, z = pg.gated_linear(x.cuda(), w.cuda(), preact=True)
    assert y.shape == (2, 3, 24) and z.shape == (2, 3, 48)
    want, _, bound, _ = forward(x.view(6, 40), w, None, "silu")
    close(y.view(6, 24), want, bound, dtype)
    dx, dw, db = pg.gated_linear_backward(y, x.cuda(), w.cuda(), z)
    assert dx.shape == (2, 3, 40) and dw.shape == (48, 40) and db.shape == (48,)
    dx, dw, db = pg.gated_linear_backward(empty(0, 9), empty(0, 5), empty(18, 5), empty(0, 18))
    assert dx.shape == (0, 5) and not dw.any() and not db.any()
    dx, dw, db = pg.gated_linear_backward(empty(7, 0), empty(7, 5), empty(0, 5), empty(7, 0))
    assert dx.shape == (7, 5) and not dx.any() and dw.shape == (0, 5)
    dx, dw, db = pg.gated_linear_backward(torch.ones(7, 3, dtype=dtype, device="cuda"), empty(7, 0), empty(6, 0),
                                          torch.ones(7, 6, dtype=dtype, device="cuda"), "relu")
    assert dx.shape == (7, 0) and dw.shape == (6, 0) and db.tolist() == [7.0] * 6


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t", [3, 150])
def test_gated_infinities_and_nan_stay_in_their_rows(dtype, t):
    n, k = 140, 200
    g = _gen(3)
    x, w = _draw(g, dtype, t, k), _draw(g, dtype, 2 * n, k)
    x[1, 7], x[2, 11] = math.inf, math.nan
    y, z = pg.gated_linear(x.cuda(), w.cuda(), act="relu", preact=True)
    want = x.double() @ w.double().t()
    assert torch.equal(torch.isfinite(z.cpu()), torch.isfinite(want))
    assert torch.equal(z[1].double().cpu(), want[1])
    assert torch.isfinite(y.cpu()).all(1).tolist() == [i not in (1, 2) for i in range(t)]


@pytest.mark.parametrize("bn,split", [(32, 0), (64, 0), (128, 0), (256, 0), (64, 3), (128, 7)])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_gated_every_tile_width_and_k_slices(dtype, bn, split):
    t, n, k = 400, 300, 1100
    g = _gen(bn + split)
    x, w, b = _draw(g, dtype, t, k), _draw(g, dtype, 2 * n, k, std=k ** -0.5), _draw(g, dtype, 2 * n)
    if bn > 32:
        pg.force_plan(bn, split)
    else:
        t = 20  # few rows: narrow tiles
        x = x[:t]
    try:
        y, z = pg.gated_linear(x.cuda(), w.cuda(), b.cuda(), "gelu", preact=True)
        again = pg.gated_linear(x.cuda(), w.cuda(), b.cuda(), "gelu")
    finally:
        pg.force_plan(0, 0)
    want, wz, bound, zb = forward(x, w, b, "gelu")
    close(y, want, bound, dtype)
    close(z, wz, zb, dtype)
    assert torch.equal(y, again)


def test_gated_half_tiles_of_a_last_wave():
    """More tiles of 256 x 128 than SM pairs by a few: the last wave's run as halves, the very
    last of them past the rows' end."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    t, n, k = 128 * (pairs + 5) - 100, 250, 1024
    g = _gen(3)
    x, w = _draw(g, torch.bfloat16, t, k), _draw(g, torch.bfloat16, 2 * n, k, std=k ** -0.5)
    pg.force_plan(128, 0)
    try:
        y = pg.gated_linear(x.cuda(), w.cuda())
    finally:
        pg.force_plan(0, 0)
    want, _, bound, _ = forward(x, w, None, "silu")
    close(y, want, bound, torch.bfloat16)


def test_gated_long_sums():
    """bfloat16 sums of more than one chunk of 16384, and float32's of several of 512."""
    for dtype, k in ((torch.bfloat16, 40000), (torch.float32, 5000)):
        g = _gen(k)
        x, w = _draw(g, dtype, 150, k), _draw(g, dtype, 260, k, std=k ** -0.5)
        y = pg.gated_linear(x.cuda(), w.cuda(), act="none")
        _, z, den = R.linear(x, w, None, "none", None)
        v, u = z[:, :130], z[:, 130:]
        # the tensor cores' truncation of long bfloat16 sums: 2^-13 of the magnitudes at most
        e = (2.0 ** -13 if dtype == torch.bfloat16 else R.NORM) * den
        close(y, v * u, v.abs() * e[:, 130:] + u.abs() * e[:, :130] + e[:, :130] * e[:, 130:], dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_gated_repeats_bitwise_on_streams_and_in_graphs(dtype):
    g = _gen(4)
    x, w = _draw(g, dtype, 200, 328).cuda(), _draw(g, dtype, 528, 328).cuda()
    x1 = x[:1]

    def work():
        y, z = pg.gated_linear(x, w, preact=True)
        return [y, z, pg.gated_linear(x1, w), pg.gated_linear(x[:20], w),
                *pg.gated_linear_backward(y, x, w, z)]

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


def test_gated_expired_wait_is_reported():
    x, w = torch.randn(300, 256, device="cuda").bfloat16(), torch.randn(400, 256, device="cuda").bfloat16()
    want = pg.gated_linear(x, w)
    limit = pg.set_wait_timeout(50_000_000)
    flags = pg.debug_flags(pg.SGEMM_DEBUG_STALL_PRODUCER)
    try:
        pg.gated_linear(x, w)
        assert pg.device_status() == pg.SGEMM_ERR_TIMEOUT
    finally:
        pg.debug_flags(flags)
        pg.set_wait_timeout(limit)
    assert torch.equal(pg.gated_linear(x, w), want) and pg.device_status() == 0


def test_gated_binding_refuses_mismatched_tensors():
    x, w = torch.randn(6, 16, device="cuda"), torch.randn(24, 16, device="cuda")
    y, z = pg.gated_linear(x, w, preact=True)
    before = pg.launch_count()
    bad = [lambda: pg.gated_linear(x, w[:23]), lambda: pg.gated_linear(x, w[:, :15]),
           lambda: pg.gated_linear(x, w, torch.randn(12, device="cuda")), lambda: pg.gated_linear(x, w, act="sine"),
           lambda: pg.gated_linear(x, w.bfloat16()), lambda: pg.gated_linear(x, w.t()),
           lambda: pg.gated_linear(x, w, out=x), lambda: pg.gated_linear(x, w, preact=y),
           lambda: pg.gated_linear_backward(y, x, w, y), lambda: pg.gated_linear_backward(z, x, w, z),
           lambda: pg.gated_linear_backward(y, x, w, None), lambda: pg.gated_linear_backward(y, x[:5], w, z)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert pg.launch_count() == before


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n", [(2000, 512), (1999, 333)])
def test_gated_bias_gradient_alone_forms_no_dz(dtype, t, n):
    """The sums alone need a workspace of their partial sums, far less than dz, and have the full
    call's bits."""
    g = _gen(t)
    x, w, dy = (_draw(g, dtype, *s).cuda() for s in ((t, 40), (2 * n, 40), (t, n)))
    z = _draw(g, dtype, t, 2 * n, std=2.0).cuda()
    want = pg.gated_linear_backward(dy, x, w, z, "gelu")[2]
    space = torch.empty(5 << 18, dtype=torch.uint8, device="cuda")
    assert space.numel() < t * 2 * n * 2
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    pg.set_workspace(space, stream=s)
    try:
        dx, dw, db = pg.gated_linear_backward(dy, x, w, z, "gelu", need_dx=False, need_dw=False, stream=s)
        s.synchronize()
    finally:
        pg.set_workspace(None, stream=s)
    assert dx is None and dw is None and torch.equal(db, want)
