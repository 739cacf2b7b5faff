"""8-bit matrices with a scale per block: their making bit for bit, and products with them
against the sums of the values they stand for in 64 bits: one row to several tiles, odd
extents, strided and unaligned rows, every activation, forced tile widths and K slices."""
import math

import pytest
import torch

import precision_gemm_gb300 as pg
from tests import _layers_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]
IDS = {torch.float32: "f32", torch.bfloat16: "bf16"}
E4M3 = torch.float8_e4m3fn


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
    fill = 0x7F if x.dtype == E4M3 else math.nan  # e4m3's NaN
    raw = torch.uint8 if x.dtype == E4M3 else x.dtype
    buf = torch.full((offset + r * (c + pad),), fill, dtype=raw, device="cuda")
    view = buf[offset:].view(r, c + pad)[:, :c]
    view.copy_(x.view(raw) if x.dtype == E4M3 else x)
    return view.view(E4M3) if x.dtype == E4M3 else view


def quantized(x, rows):
    """q and scales by the definition, in float32 on the CPU, a block at a time."""
    x = x.float()
    t, k = x.shape
    q, scales = torch.empty(t, k, dtype=E4M3), torch.empty(-(-t // rows), -(-k // 128))
    for i in range(0, t, rows):
        for j in range(0, k, 128):
            b = x[i:i + rows, j:j + 128]
            s = torch.clamp_min(b.abs().max() / torch.tensor(448.0), torch.finfo(torch.float32).tiny)
            scales[i // rows, j // 128] = s
            q[i:i + rows, j:j + 128] = (b / s).to(E4M3)
    return q, scales


def values(q, scales, rows):
    """The values that an 8-bit matrix stands for, in 64 bits."""
    t, k = q.shape
    spread = scales.double().repeat_interleave(rows, 0)[:t].repeat_interleave(128, 1)[:, :k]
    return q.float().double() * spread


def _bits(x):
    return x.cpu().contiguous().view(torch.uint8 if x.dtype == E4M3 else torch.int32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("t,k", [(1, 1), (3, 127), (2, 128), (5, 129), (130, 300), (260, 777), (128, 1024), (40, 4096)])
def test_quantize(dtype, rows, t, k):
    g = _gen(t + k)
    # spreads from far below to far above one, so that scales differ from block to block
    x = (_draw(g, torch.float32, t, k) * torch.exp2(torch.randint(-20, 20, (t, 1), generator=g).float())).to(dtype)
    q, scales = pg.quantize(x.cuda(), rows)
    wq, ws = quantized(x, rows)
    assert q.dtype == E4M3 and q.shape == x.shape and q.stride(0) % 16 == 0
    assert torch.equal(_bits(scales), _bits(ws)) and torch.equal(_bits(q), _bits(wq))


def test_quantize_every_bfloat16_quotient():
    """All 2^16 bfloat16 numbers but NaN and infinities, in blocks of their own magnitude and under
    a large neighbour: ties, subnormal results, the smallest scale."""
    u = torch.arange(0x7F80, dtype=torch.int32)
    x = torch.cat([u, u | 0x8000]).to(torch.int16).view(torch.bfloat16)
    near = x.view(-1, 128)
    far = x.clone().view(-1, 64)
    far = torch.cat([far, far.roll(1, 0)], 1)
    for m in (near, far):
        q, scales = pg.quantize(m.cuda())
        wq, ws = quantized(m, 1)
        assert torch.equal(_bits(scales), _bits(ws)) and torch.equal(_bits(q), _bits(wq))


def test_quantize_random_quotients():
    """Two million float32 numbers of every magnitude, some blocks with values far below their
    largest, against the divisions of the definition."""
    g = _gen(8)
    for dtype in DTYPES:
        x = torch.randn(2048, 1024, generator=g)
        x *= torch.exp2(torch.randint(-120, 120, (2048, 8), generator=g).float()).repeat_interleave(128, 1)
        x = torch.where(torch.rand(x.shape, generator=g) < 0.05, x * 2.0 ** -20, x).to(dtype)
        q, scales = pg.quantize(x.cuda())
        b = x.float().view(2048, 8, 128)
        ws = torch.clamp_min(b.abs().amax(2) / torch.tensor(448.0), torch.finfo(torch.float32).tiny)
        wq = (b / ws[:, :, None]).to(E4M3).view(2048, 1024)
        assert torch.equal(_bits(scales), _bits(ws)) and torch.equal(_bits(q), _bits(wq))


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_zeros_infinities_nan_and_strides(rows):
    x = torch.randn(140, 400, generator=_gen(2))
    x[0, :128] = 0
    x[1, 130], x[2, 300] = math.inf, math.nan
    x[130:, 384:] = 0
    q, scales = pg.quantize(_strided(x, 3, 1), rows)
    wq, ws = quantized(x, rows)
    assert torch.equal(torch.isnan(scales.cpu()), torch.isnan(ws))
    assert torch.equal(torch.nan_to_num(scales.cpu()), torch.nan_to_num(ws))
    assert torch.equal(torch.isnan(q.cpu().float()), torch.isnan(wq.float()))
    assert torch.equal(torch.nan_to_num(q.cpu().float()), torch.nan_to_num(wq.float()))
    if rows == 1:
        assert scales[0, 0] == 2.0 ** -126 and scales[1, 1] == math.inf and math.isnan(scales[2, 2])
    q3, s3 = pg.quantize(torch.randn(2, 3, 200, device="cuda"))
    assert q3.shape == (2, 3, 200) and s3.shape == (2, 3, 2)
    q0, s0 = pg.quantize(torch.empty(0, 200, device="cuda"), rows)
    assert q0.shape == (0, 200) and s0.shape == (0, 2)


def product(xq, xs, wq, ws, bias, name, residual):
    """y, and the sums of its terms' magnitudes, of matrices as they are stored."""
    x, w = values(xq, xs, 1), values(wq, ws, 128)
    return R.linear(x, w, bias, name, residual)[::2]


def _weights(g, n, k):
    q, s = pg.quantize(_draw(g, torch.float32, n, k, std=k ** -0.5).cuda(), 128)
    return q, s


SIZES = [(1, 1, 1), (1, 130, 3), (1, 4096, 512), (2, 64, 128), (5, 1000, 777), (17, 257, 129), (33, 640, 256),
         (128, 128, 1024), (130, 300, 777), (257, 513, 1000), (300, 256, 65), (1500, 300, 777), (600, 1030, 4100)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k", SIZES)
def test_block_linear(dtype, t, n, k):
    g = _gen(t * 7 + n * 3 + k)
    x = _draw(g, dtype, t, k)
    b, r = _draw(g, dtype, n), _draw(g, dtype, t, n)
    w, s = _weights(g, n, k)
    name = R.ACTS[(t + n + k) % 5]
    y = pg.block_linear(x.cuda(), w, s, b.cuda(), name, r.cuda())
    xq, xs = pg.quantize(x.cuda())
    want, den = product(xq.cpu(), xs.cpu(), w.cpu(), s.cpu(), b, name, r)
    R.close(y, want, den, dtype)
    # x in 8 bits already
    again = pg.block_linear(xq, w, s, b.cuda(), name, r.cuda(), x_scales=xs, dtype=dtype)
    assert torch.equal(y, again)
    y = pg.block_linear(x.cuda(), w, s)
    want, den = product(xq.cpu(), xs.cpu(), w.cpu(), s.cpu(), None, "none", None)
    R.close(y, want, den, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("t", [2, 200])
def test_block_activations_over_their_range(dtype, name, t):
    n, k = 192, 32
    g = _gen(5)
    x, b = _draw(g, dtype, t, k), torch.linspace(-12, 12, n).to(dtype)
    x[0] = 0
    w, s = _weights(g, n, k)
    y = pg.block_linear(x.cuda(), w, s, b.cuda(), name)
    want, den = product(*(v.cpu() for v in pg.quantize(x.cuda())), w.cpu(), s.cpu(), b, name, None)
    R.close(y, want, den, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k,pad,offset", [(2, 70, 100, 3, 1), (140, 200, 136, 5, 3), (140, 200, 136, 8, 8),
                                              (300, 136, 256, 16, 16), (300, 130, 64, 1, 0), (1, 64, 72, 7, 2)])
def test_block_strides_and_alignment(dtype, t, n, k, pad, offset):
    g = _gen(t + pad)
    x, b, r = _draw(g, dtype, t, k), _draw(g, dtype, n), _draw(g, dtype, t, n)
    w, s = _weights(g, n, k)
    out = _strided(torch.zeros(t, n, dtype=dtype), pad, offset)
    ws, ss = _strided(w, pad, offset), _strided(s, pad, offset)
    got = pg.block_linear(_strided(x, pad, offset), ws, ss, b.cuda(), "silu", _strided(r, pad, offset), out=out)
    assert got is out
    xq, xs = pg.quantize(x.cuda())
    want, den = product(xq.cpu(), xs.cpu(), w.cpu(), s.cpu(), b, "silu", r)
    R.close(out, want, den, dtype)
    gaps = out.as_strided((t, pad), (n + pad, 1), offset + n)[:t - 1]
    assert torch.isnan(gaps).all()
    y = pg.block_linear(_strided(xq, pad, offset), ws, ss, b.cuda(), "silu", r.cuda(),
                        x_scales=_strided(xs, pad, offset), dtype=dtype)
    assert torch.equal(y, out)
    both = r.cuda()
    assert pg.block_linear(x.cuda(), w, s, b.cuda(), "silu", both, out=both) is both
    assert torch.equal(both, y)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t,n,k", [(1, 300, 256), (7, 333, 500), (40, 96, 2048), (300, 520, 256), (300, 77, 300)])
def test_block_residual_in_place(dtype, t, n, k):
    """residual and out may be the same tensor, in every kernel that finishes a product."""
    g = _gen(t + n)
    x, r = _draw(g, dtype, t, k).cuda(), _draw(g, dtype, t, n).cuda()
    w, s = _weights(g, n, k)
    want = pg.block_linear(x, w, s, act="silu", residual=r)
    assert pg.block_linear(x, w, s, act="silu", residual=r, out=r) is r
    assert torch.equal(r, want)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("n,k", [(333, 500), (40, 1030), (1100, 4096), (128, 16)])
@pytest.mark.parametrize("t", [2, 7, 8, 9, 15, 16, 17])
def test_block_few_rows(dtype, t, n, k):
    """Around the numbers of rows where kernels change."""
    g = _gen(t + n)
    x, b, r = _draw(g, dtype, t, k), _draw(g, dtype, n), _draw(g, dtype, t, n)
    w, s = _weights(g, n, k)
    y = pg.block_linear(x.cuda(), w, s, b.cuda(), "gelu", r.cuda())
    q, xs = quantized(x, 1)
    want, _, den = R.linear(values(q, xs, 1), values(w.cpu(), s.cpu(), 128), b, "gelu", r)
    R.close(y, want, den, dtype)
    assert torch.equal(pg.block_linear(q.cuda(), w, s, b.cuda(), "gelu", r.cuda(), xs.cuda(), dtype=dtype), y)


def test_block_scales_meet_their_blocks():
    """Every block's scale a power of two of its own and small whole numbers as values: each sum
    is exact, so a scale at another block shows."""
    t, n, k = 300, 520, 700
    g = _gen(9)
    xq = torch.randint(-3, 4, (t, k), generator=g).float().to(E4M3)
    wq = torch.randint(-3, 4, (n, k), generator=g).float().to(E4M3)
    xs = torch.exp2(torch.randint(-2, 3, (t, 6), generator=g).float())
    ws = torch.exp2(torch.randint(-2, 3, (5, 6), generator=g).float())
    want = values(xq, xs, 1) @ values(wq, ws, 128).t()
    for tt in (1, 20, t):
        y = pg.block_linear(xq[:tt].cuda(), wq.cuda(), ws.cuda(), x_scales=xs[:tt].cuda(), dtype=torch.float32)
        assert torch.equal(y.double().cpu(), want[:tt])


def test_block_sums_are_float32():
    """Results whose terms cancel to 2^-20 of them: a tensor core that kept fewer bits of a block's
    sum than FP32 does would lose them.  The products are whole numbers, their sums below 2^24."""
    t, n, k = 130, 200, 512
    g = _gen(12)
    x = torch.randint(0, 2, (t, k), generator=g).float() * 448
    w = torch.randint(0, 2, (n, k), generator=g).float() * 448
    x[:, ::7], w[:, ::5] = 1, -1
    xs, ws = torch.ones(t, 4), torch.ones(2, 4)
    want = x.double() @ w.double().t()
    y = pg.block_linear(x.to(E4M3).cuda(), w.to(E4M3).cuda(), ws.cuda(), x_scales=xs.cuda(), dtype=torch.float32)
    den = x.double().abs() @ w.double().abs().t()
    R.close(y, want, den, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
@pytest.mark.parametrize("t", [3, 150])
def test_block_infinities_and_nan_stay_in_their_rows(dtype, t):
    g = _gen(3)
    x = _draw(g, dtype, t, 200)
    x[1, 7], x[2, 150] = math.inf, math.nan
    w, s = _weights(g, 140, 200)
    y = pg.block_linear(x.cuda(), w, s).cpu()
    assert torch.isnan(y).all(1).tolist() == [i in (1, 2) for i in range(t)]
    assert torch.isfinite(y).all(1).tolist() == [i not in (1, 2) for i in range(t)]


@pytest.mark.parametrize("bn,split", [(64, 0), (128, 0), (256, 0), (64, 3), (128, 9), (256, 2)])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_block_every_tile_width_and_k_slices(dtype, bn, split):
    t, n, k = 400, 600, 1100
    g = _gen(bn + split)
    x, b, r = _draw(g, dtype, t, k), _draw(g, dtype, n), _draw(g, dtype, t, n)
    w, s = _weights(g, n, k)
    pg.force_plan(bn, split)
    try:
        y = pg.block_linear(x.cuda(), w, s, b.cuda(), "gelu", r.cuda())
        again = pg.block_linear(x.cuda(), w, s, b.cuda(), "gelu", r.cuda())
    finally:
        pg.force_plan(0, 0)
    want, den = product(*(v.cpu() for v in pg.quantize(x.cuda())), w.cpu(), s.cpu(), b, "gelu", r)
    R.close(y, want, den, dtype)
    assert torch.equal(y, again)


def test_block_more_tiles_than_a_wave():
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    t, n, k = 256 * (pairs + 5) - 200, 250, 512
    g = _gen(3)
    x = _draw(g, torch.bfloat16, t, k)
    w, s = _weights(g, n, k)
    y = pg.block_linear(x.cuda(), w, s, act="relu")
    want, den = product(*(v.cpu() for v in pg.quantize(x.cuda())), w.cpu(), s.cpu(), None, "relu", None)
    R.close(y, want, den, torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS.get)
def test_block_empty_extents_and_leading_dimensions(dtype):
    g = _gen(1)
    b, r = _draw(g, dtype, 9), _draw(g, dtype, 4, 9)
    w, s = pg.quantize(torch.empty(9, 0, device="cuda"), 128)
    y = pg.block_linear(torch.empty(4, 0, dtype=dtype, device="cuda"), w, s, b.cuda(), "silu", r.cuda())
    want, _, den = R.linear(torch.zeros(4, 0), torch.zeros(9, 0), b, "silu", r)
    R.close(y, want, den, dtype)
    w, s = _weights(g, 24, 200)
    assert pg.block_linear(torch.empty(0, 200, dtype=dtype, device="cuda"), w, s).shape == (0, 24)
    x = _draw(g, dtype, 2, 3, 200).cuda()
    y = pg.block_linear(x, w, s)
    assert y.shape == (2, 3, 24)
    assert torch.equal(y.view(6, 24), pg.block_linear(x.view(6, 200), w, s))
    xq, xs = pg.quantize(x)
    assert torch.equal(y, pg.block_linear(xq, w, s, x_scales=xs, dtype=dtype))


@pytest.mark.parametrize("k", [0, 16, 130, 700])
def test_block_bias_of_many_tiles(k):
    """Several tiles to a thread block one after another, few or no blocks of k in each: every tile
    gets its own columns' bias."""
    t, n, dtype = 700, 9000, torch.bfloat16
    g = _gen(k)
    x, b, r = _draw(g, dtype, t, k), _draw(g, dtype, n), _draw(g, dtype, t, n)
    if k:
        w, s = _weights(g, n, k)
    else:
        w, s = pg.quantize(torch.empty(n, 0, device="cuda"), 128)
    pg.force_plan(64, 1)
    try:
        y = pg.block_linear(x.cuda(), w, s, b.cuda(), "relu", r.cuda())
    finally:
        pg.force_plan()
    if k:
        want, _, den = R.linear(values(*quantized(x, 1), 1), values(w.cpu(), s.cpu(), 128), b, "relu", r)
    else:
        want, _, den = R.linear(torch.zeros(t, 0), torch.zeros(n, 0), b, "relu", r)
    R.close(y, want, den, dtype)


def test_block_repeats_bitwise_on_streams_and_in_graphs():
    g = _gen(4)
    x = _draw(g, torch.bfloat16, 300, 1000).cuda()
    w, s = _weights(g, 500, 1000)

    def work():
        q, qs = pg.quantize(x)
        return [qs, pg.block_linear(x, w, s), pg.block_linear(x[:1], w, s, act="gelu"), pg.block_linear(x[:40], w, s),
                pg.block_linear(q, w, s, x_scales=qs)]

    first = work()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = work()
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        held = work()
    for v in held:
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_block_expired_wait_is_reported():
    g = _gen(5)
    x = _draw(g, torch.bfloat16, 300, 512).cuda()
    w, s = _weights(g, 400, 512)
    want = pg.block_linear(x, w, s)
    limit = pg.set_wait_timeout(50_000_000)
    flags = pg.debug_flags(pg.SGEMM_DEBUG_STALL_PRODUCER)
    try:
        pg.block_linear(x, w, s)
        assert pg.device_status() == pg.SGEMM_ERR_TIMEOUT
    finally:
        pg.debug_flags(flags)
        pg.set_wait_timeout(limit)
    assert torch.equal(pg.block_linear(x, w, s), want) and pg.device_status() == 0


def test_block_binding_refuses_mismatched_tensors():
    x = torch.randn(6, 200, device="cuda")
    w, s = pg.quantize(torch.randn(140, 200, device="cuda"), 128)
    xq, xs = pg.quantize(x)
    before = pg.launch_count()
    bad = [lambda: pg.block_linear(x, w.view(torch.uint8), s), lambda: pg.block_linear(x, w.float(), s),
           lambda: pg.block_linear(x, w[:, :199], s), lambda: pg.block_linear(x, w, s[:1]),
           lambda: pg.block_linear(x, w, s.double()), lambda: pg.block_linear(x, w, s.t()),
           lambda: pg.block_linear(x.half(), w, s), lambda: pg.block_linear(xq, w, s),
           lambda: pg.block_linear(x, w, s, x_scales=xs), lambda: pg.block_linear(xq, w, s, x_scales=xs[:5]),
           lambda: pg.block_linear(x, w, s, dtype=torch.bfloat16), lambda: pg.block_linear(x, w, s, act="sine"),
           lambda: pg.block_linear(xq, w, s, x_scales=xs, dtype=torch.float16),
           lambda: pg.block_linear(xq, w, s, torch.randn(140, device="cuda"), x_scales=xs),
           lambda: pg.block_linear(x, w, s, out=x), lambda: pg.quantize(x.double()), lambda: pg.quantize(x.t()),
           lambda: pg.quantize(x.view(2, 3, 200), 128)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pg.SgemmError):
        pg.quantize(x, 64)
    assert pg.launch_count() == before


def _e4m3(g, *shape):
    """Every finite value as likely as the next."""
    v = torch.randint(0, 255, shape, generator=g, dtype=torch.uint8)
    return torch.where(v % 128 == 127, v - 1, v).view(E4M3)


@pytest.mark.parametrize("power", [-63, 40])
@pytest.mark.parametrize("t", [1, 9, 40, 300])
def test_block_scales_up_to_their_stated_range(t, power):
    """Products of two scales from the smallest normal floats on, and large ones: all their bits count."""
    n, k = 200, 700
    g = _gen(t)
    xq, wq = _e4m3(g, t, k), _e4m3(g, n, k)
    xs, ws = (torch.exp2(power + torch.rand(s, generator=g)) for s in ((t, 6), (2, 6)))
    y = pg.block_linear(xq.cuda(), wq.cuda(), ws.cuda(), x_scales=xs.cuda(), dtype=torch.float32).double().cpu()
    want, den = product(xq, xs, wq, ws, None, "none", None)
    assert ((y - want).abs() <= R.NORM * den).all(), float(((y - want).abs() / den).max())


@pytest.mark.parametrize("mixed", [False, True], ids=["halves", "mixed"])
@pytest.mark.parametrize("t", [1, 9, 40, 130])
def test_block_sums_keep_what_cancels(t, mixed):
    """In each block of 128, 60 terms of 448^2, 60 of -448^2 and eight small ones: whole numbers whose
    partial sums stay below 2^24 in any order, so a sum in FP32 is exact, while one that is cut to 22 bits
    after every 32 k is not.  Every element has to be equal."""
    n, k = 200, 512
    g = _gen(t)
    x, w = torch.full((t, 4, 128), 448.0), torch.full((n, 4, 128), 448.0)
    x[1::2] *= -1
    for b in range(4):
        at = torch.randperm(128, generator=g) if mixed else torch.arange(128)
        small = at[torch.arange(7, 128, 16)]
        large = at[torch.arange(128) % 16 != 7]
        x[:, b, small] = torch.randint(1, 4, (t, 8), generator=g).float()
        w[:, b, small] = torch.randint(-3, 4, (n, 8), generator=g).float()
        w[:, b, large[60:]] *= -1
    assert (x.abs().double().view(t, k) @ w.abs().double().view(n, k).t()).max() / 8 < 2 ** 24  # a half of a block's
    want = x.double().view(t, k) @ w.double().view(n, k).t()
    cut = torch.zeros(t, n, dtype=torch.float64)
    for b in range(4):
        s = torch.zeros(t, n, dtype=torch.float64)
        for c in range(0, 128, 32):
            s += x[:, b, c:c + 32].double() @ w[:, b, c:c + 32].double().t()
            step = torch.exp2(torch.floor(torch.log2(s.abs().clamp_min(1))) - 21)
            s = torch.trunc(s / step) * step
        cut += s
    assert mixed or not torch.equal(cut, want)
    y = pg.block_linear(x.view(t, k).to(E4M3).cuda(), w.view(n, k).to(E4M3).cuda(), torch.ones(2, 4, device="cuda"),
                        x_scales=torch.ones(t, 4, device="cuda"), dtype=torch.float32)
    assert torch.equal(y.double().cpu(), want)
