"""The example's gated block: the layer calls chained as they are used.  Its gradients
against differences of its definition in 64 bits, training and serving in 8 bits, and
the chain in captured graphs, on several threads and over given workspaces."""
import os
import sys
import threading

import pytest
import torch

import precision_gemm_gb300 as pg
from tests import _layers_ref as R
from tests import test_block_gpu as TB
from tests import test_gated_gpu as TG
from tests import test_norm_gpu as TN

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gated_feed_forward as gf  # noqa: E402

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


def _block(width, hidden, act, dtype, seed):
    block = gf.GatedFeedForward(width, hidden, act, dtype, seed)
    gen = torch.Generator().manual_seed(seed + 100)
    for name in ("norm", "shift", "b1", "b2"):  # ones and zeros would hide a mistake
        p = block.params[name]
        block.params[name] = (torch.randn(p.shape, generator=gen) * 0.5 + (name == "norm")).to(dtype).cuda()
    return block


def _block64(x, p, act):
    mean = x.mean(1, keepdim=True)
    h = (x - mean) * ((x - mean).square().mean(1, keepdim=True) + 1e-5).rsqrt() * p["norm"] + p["shift"]
    z = h @ p["w1"].t() + p["b1"]
    n = z.shape[1] // 2
    return x + (R.act(z[:, :n], act) * z[:, n:]) @ p["w2"].t() + p["b2"]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,width,hidden", [(50, 24, 40), (3, 130, 65), (140, 64, 200)])
def test_block_gradients_against_differences(tokens, width, hidden, act):
    """Directional differences in 64 bits, step 1e-5: their error is of order 1e-9 of the loss.
    The gradients come through two to four products of FP32 sums one after another, each within
    1e-5 of its terms' magnitudes."""
    block = _block(width, hidden, act, torch.float32, 3)
    gen = torch.Generator().manual_seed(4)
    x, dy = torch.randn(tokens, width, generator=gen), torch.randn(tokens, width, generator=gen)
    y, saved = block.forward(x.cuda())
    at = {k: v.double().cpu() for k, v in block.params.items()}
    want = _block64(x.double(), at, act)
    assert float((y.double().cpu() - want).norm() / want.norm()) < 2e-5
    dx, grads = block.backward(dy.cuda(), saved)

    def loss(x, params):
        return float((_block64(x, params, act) * dy.double()).sum())

    h = 1e-5
    for name, grad in [("x", dx), *grads.items()]:
        u = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
        sides = []
        for s in (h, -h):
            moved = dict(at)
            if name != "x":
                moved[name] = at[name] + s * u
            sides.append(loss(x.double() + (s * u if name == "x" else 0.0), moved))
        diff = (sides[0] - sides[1]) / (2 * h)
        grad = grad.double().cpu()
        assert abs(diff - float((grad * u).sum())) <= 5e-5 * float((grad.abs() * u.abs()).sum()), name


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("tokens", [1, 7, 200])
def test_block_step_by_step(dtype, tokens):
    """Every call of the chain, forward and backward, within its own bound for the inputs it got."""
    width, hidden, act = 200, 264, "gelu_tanh"
    block = _block(width, hidden, act, dtype, 5)
    p = {k: v.cpu() for k, v in block.params.items()}
    gen = torch.Generator().manual_seed(6)
    x, dy = (torch.randn(tokens, width, generator=gen).to(dtype) for _ in range(2))
    y, (_, mean, rstd, h, z, a) = block.forward(x.cuda())
    dx, grads = block.backward(dy.cuda(), (x.cuda(), mean, rstd, h, z, a))
    hc, zc, ac = h.cpu(), z.cpu(), a.cpu()
    want, den = TN.forward(x, p["norm"], p["shift"], 1e-5)
    TN.close(h, want[0], den[0], dtype)
    wy, wz, bound, zbound = TG.forward(hc, p["w1"], p["b1"], act)
    TG.close(a, wy, bound, dtype)
    TG.close(z, wz, zbound, dtype)
    want, _, den = R.linear(ac, p["w2"], p["b2"], "none", x)
    R.close(y, want, den, dtype)
    da = pg.linear_backward(dy.cuda(), a, block.params["w2"])[0]
    dh = pg.gated_linear_backward(da, h, block.params["w1"], z, act)[0]
    want, den = TG.backward(da.cpu(), hc, p["w1"], act, zc)
    TG._check_backward((dh, grads["w1"], grads["b1"]), want, den, dtype)
    want, den = TN.backward(dh.cpu(), x, p["norm"], mean.cpu(), rstd.cpu(), dy)
    for got, w, d in zip((dx, grads["norm"], grads["shift"]), want, den):
        TN.close(got, w, d, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("tokens", [1, 5, 150])
def test_served_block(dtype, tokens):
    """The served block's last product within its bound for the inputs it got, from 8-bit values
    that the definition gives bit for bit."""
    width, hidden, act = 200, 264, "silu"
    block = _block(width, hidden, act, dtype, 9)
    served = gf.Served(block)
    x = torch.randn(tokens, width, generator=torch.Generator().manual_seed(2)).to(dtype)
    y = served.forward(x.cuda())
    h = pg.layer_norm(x.cuda(), served.norm, served.shift)
    q, s = pg.quantize(h)
    want_q, want_s = TB.quantized(h.cpu(), 1)
    assert torch.equal(TB._bits(q), TB._bits(want_q)) and torch.equal(s.cpu(), want_s)
    parts = []
    for w, bias, name in ((served.gate, served.bg, act), (served.up, served.bu, "none")):
        got = pg.block_linear(q, *w, bias, name, x_scales=s, dtype=dtype)
        want, _, den = R.linear(TB.values(want_q, want_s, 1), TB.values(w[0].cpu(), w[1].cpu(), 128), bias.cpu(), name, None)
        R.close(got, want, den, dtype)
        parts.append(got)
    m = (parts[0] * parts[1]).cpu()
    wq, ws = TB.quantized(m, 1)
    dq, ds = TB.quantized(block.params["w2"].cpu(), 128)
    want, _, den = R.linear(TB.values(wq, ws, 1), TB.values(dq, ds, 128), served.b2.cpu(), "none", x)
    R.close(y, want, den, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_example_runs(dtype):
    teacher, block = gf.GatedFeedForward(128, 256, dtype=dtype, seed=7), gf.GatedFeedForward(128, 256, dtype=dtype, seed=8)
    losses = gf.train(block, teacher, 256, 128, 4)
    assert all(0 < v < float("inf") for v in losses)
    x = torch.randn(64, 128, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    assert torch.isfinite(gf.Served(block).forward(x)).all()


def _chain(block, served, x, dy):
    y, saved = block.forward(x)
    dx, grads = block.backward(dy, saved)
    return [y, dx, *grads.values(), served.forward(x), served.forward(x[:1])]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_two_graphs_of_the_block_share_a_workspace(dtype):
    """Training steps of two sizes captured on one stream, replayed in turn, with an eager step
    of the same parameters between them."""
    block = _block(136, 260, "silu", dtype, 1)
    served = gf.Served(block)
    gen = torch.Generator().manual_seed(3)
    cases = [[torch.randn(t, 136, generator=gen).to(dtype).cuda() for _ in range(2)] for t in (190, 33)]
    want = [_chain(block, served, *c) for c in cases]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for c in cases:
            _chain(block, served, *c)  # sizes the stream's workspace
    s.synchronize()
    graphs, held = [], []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            held.append(_chain(block, served, *c))
        graphs.append(graph)
    for order in ((0, 1, 0), (1, 1, 0)):
        for i in order:
            for v in held[i]:
                v.zero_()
            graphs[i].replay()
            eager = _chain(block, served, *cases[1 - i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held[i], want[i]))
            assert all(torch.equal(a, b) for a, b in zip(eager, want[1 - i]))


def test_blocks_on_several_threads():
    """Four host threads, each on a stream of its own, with different sizes and types."""
    jobs, errors = [], []
    for i, (t, width, hidden, dtype) in enumerate([(190, 136, 260, torch.float32), (5, 512, 700, torch.bfloat16),
                                                   (300, 77, 131, torch.bfloat16), (1, 1024, 520, torch.float32)]):
        block = _block(width, hidden, "gelu", dtype, i)
        gen = torch.Generator().manual_seed(i)
        x, dy = (torch.randn(t, width, generator=gen).to(dtype).cuda() for _ in range(2))
        served = gf.Served(block)
        jobs.append((block, served, x, dy, _chain(block, served, x, dy)))
    torch.cuda.synchronize()

    def run(block, served, x, dy, want):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = _chain(block, served, x, dy)
                    s.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_given_workspaces(dtype):
    """Over a workspace full of NaN every call gives what it gave; over one that is too small it
    fails with the library's error and launches nothing."""
    block = _block(777, 300, "gelu", dtype, 1)
    gen = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(150, 777, generator=gen).to(dtype).cuda() for _ in range(2))
    p = block.params
    w8, s8 = pg.quantize(p["w1"], 128)
    h, mean, rstd = pg.layer_norm(x, p["norm"], p["shift"], stats=True)
    a, z = pg.gated_linear(h, p["w1"], p["b1"], "gelu", preact=True)
    calls = [lambda s=None: pg.layer_norm_backward(dy, x, p["norm"], mean, rstd, stream=s),
             lambda s=None: pg.gated_linear(h, p["w1"], p["b1"], "gelu", preact=True, stream=s),
             lambda s=None: pg.gated_linear_backward(a, h, p["w1"], z, "gelu", stream=s),
             lambda s=None: (pg.block_linear(h, w8, s8, p["b1"], "relu", stream=s),),
             lambda s=None: (pg.block_linear(h[:8], w8, s8, p["b1"], "relu", stream=s),)]
    want = [c() for c in calls]
    space = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    try:
        for call, w in zip(calls, want):
            space.fill_(255)
            torch.cuda.synchronize()
            pg.set_workspace(space, stream=s)
            got = call(s)
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(got, w))
            pg.set_workspace(small, stream=s)
            before = pg.launch_count()
            with pytest.raises(pg.SgemmError) as e:
                call(s)
            assert e.value.code == pg.SGEMM_ERR_WORKSPACE and pg.launch_count() == before
    finally:
        pg.set_workspace(None, stream=s)


def test_large_offsets():
    """Rows that start beyond 2^31 elements: of x in a gated layer and its gradients, of x and of
    the weights in an 8-bit product."""
    t, k, n = 2 ** 20 + 7, 2100, 20
    dtype = torch.bfloat16
    gen = torch.Generator().manual_seed(1)
    x = torch.zeros(t, k, dtype=dtype, device="cuda")
    tail = torch.randn(5, k, generator=gen).to(dtype)
    x[-5:] = tail.cuda()
    w = (torch.randn(2 * n, k, generator=gen) * k ** -0.5).to(dtype)
    y, z = pg.gated_linear(x, w.cuda(), preact=True)
    wy, wz, bound, zbound = TG.forward(tail, w, None, "silu")
    TG.close(y[-5:], wy, bound, dtype)
    TG.close(z[-5:], wz, zbound, dtype)
    assert not y[:-5].any()
    dy = torch.zeros(t, n, dtype=dtype, device="cuda")
    dtail = torch.randn(5, n, generator=gen).to(dtype)
    dy[-5:] = dtail.cuda()
    dx, dw, db = pg.gated_linear_backward(dy, x, w.cuda(), z)
    want, den = TG.backward(dtail, tail, w, "silu", z[-5:].cpu())
    TG._check_backward((dx[-5:], dw, db), want, den, dtype)
    assert not dx[:-5].any()
    del dx, dw, db, dy, y, z
    w8, s8 = pg.quantize(w.cuda(), 128)
    y = pg.block_linear(x, w8, s8)
    xv = TB.values(*TB.quantized(tail, 1), 1)
    want, _, den = R.linear(xv, TB.values(w8.cpu(), s8.cpu(), 128), None, "none", None)
    R.close(y[-5:], want, den, dtype)
    assert not y[:-5].any()
    # ... and as weights, whose last block of 128 rows holds the tail
    w8, s8 = pg.quantize(x, 128)
    del x
    first = t - t % 128
    rows = torch.zeros(t % 128, k, dtype=dtype)
    rows[-5:] = tail
    wv = TB.values(*TB.quantized(rows, 128), 128)
    assert first % 128 == 0 and not s8[:-1].gt(torch.finfo(torch.float32).tiny).any()
    for m in (1, 40):
        v = torch.randn(m, k, generator=gen).to(dtype)
        y = pg.block_linear(v.cuda(), w8, s8)
        want, _, den = R.linear(TB.values(*TB.quantized(v, 1), 1), wv, None, "none", None)
        R.close(y[:, first:], want, den, dtype)
        assert not y[:, :first].any()
