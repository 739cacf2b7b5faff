"""Refusals of the layer calls that need no GPU: the library names the first
invalid argument before it touches a device, and the binding refuses tensors it
cannot pass."""
import pytest
import torch

import precision_gemm_gb300 as pg
from precision_gemm_gb300 import build as pgbuild

P = 4096  # an address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    pgbuild.build()
    return pg.load_library()


NAMES = {
    "sgemm_linear": "dtype t n k x ldx w ldw bias act residual ldr y ldy preact ldz stream",
    "sgemm_linear_backward": "dtype t n k dy lddy x ldx w ldw act preact ldz dx lddx dw lddw dbias stream",
    "sgemm_route": "dtype tokens experts top logits ldl score balance groups group_top renormalize scale mask weights "
                   "ids stream",
    "sgemm_route_backward": "dtype tokens experts top dweights logits ldl ids score renormalize scale dlogits lddl "
                            "stream",
    "sgemm_expert_plan": "tokens top experts ids counts offsets rows slots stream",
    "sgemm_expert_linear": "dtype tokens top experts n k gather x ldx w ldw stride_w bias act offsets rows y ldy "
                           "preact ldz stream",
    "sgemm_expert_linear_backward": "dtype tokens top experts n k gather dy lddy x ldx w ldw stride_w act preact ldz "
                                    "offsets rows slots dx lddx dw lddw stride_dw dbias stream",
    "sgemm_expert_combine": "dtype tokens top n x ldx slots weights residual ldr y ldy stream",
    "sgemm_expert_combine_backward": "dtype tokens top n dy lddy x ldx rows slots weights dx lddx dweights stream",
}
GOOD = dict(dtype=0, t=4, n=24, k=16, tokens=4, top=2, experts=8, gather=1, score=0, groups=2, group_top=1,
            renormalize=1, scale=1.0, act=2, stream=None, ldx=16, ldw=16, ldr=24, ldy=24, ldz=24, lddy=24, lddx=16,
            lddw=16, ldl=8, lddl=8, stride_w=24 * 16, stride_dw=24 * 16)


def _call(lib, name, **bad):
    args = dict(GOOD)
    if name.startswith("sgemm_expert_combine"):
        args.update(ldx=24, lddx=24)
    args.update(bad)
    return getattr(lib, name)(*[args.get(a, P) for a in NAMES[name].split()])


BAD = [
    ("sgemm_linear", "dtype", 2), ("sgemm_linear", "t", -1), ("sgemm_linear", "n", 2 ** 31), ("sgemm_linear", "k", -1),
    ("sgemm_linear", "x", None), ("sgemm_linear", "ldx", 15), ("sgemm_linear", "w", None), ("sgemm_linear", "ldw", 0),
    ("sgemm_linear", "act", 5), ("sgemm_linear", "ldr", 23), ("sgemm_linear", "y", None), ("sgemm_linear", "ldy", 23),
    ("sgemm_linear", "ldz", 3),
    ("sgemm_linear_backward", "dtype", -1), ("sgemm_linear_backward", "dy", None), ("sgemm_linear_backward", "lddy", 1),
    ("sgemm_linear_backward", "x", None), ("sgemm_linear_backward", "w", None), ("sgemm_linear_backward", "act", -1),
    ("sgemm_linear_backward", "preact", None), ("sgemm_linear_backward", "lddx", 15),
    ("sgemm_linear_backward", "lddw", 15),
    ("sgemm_route", "experts", 0), ("sgemm_route", "experts", 513), ("sgemm_route", "top", 0), ("sgemm_route", "top", 9),
    ("sgemm_route", "logits", None), ("sgemm_route", "ldl", 7), ("sgemm_route", "score", 2), ("sgemm_route", "groups", 3),
    ("sgemm_route", "groups", 0), ("sgemm_route", "group_top", 3), ("sgemm_route", "group_top", 0),
    ("sgemm_route", "renormalize", 2), ("sgemm_route", "scale", float("nan")), ("sgemm_route", "weights", None),
    ("sgemm_route", "ids", None),
    ("sgemm_route_backward", "dweights", None), ("sgemm_route_backward", "ids", None),
    ("sgemm_route_backward", "score", -1), ("sgemm_route_backward", "scale", float("inf")),
    ("sgemm_route_backward", "dlogits", None), ("sgemm_route_backward", "lddl", 1),
    ("sgemm_expert_plan", "tokens", -1), ("sgemm_expert_plan", "tokens", 2 ** 30), ("sgemm_expert_plan", "top", 33),
    ("sgemm_expert_plan", "experts", 600), ("sgemm_expert_plan", "ids", None), ("sgemm_expert_plan", "counts", None),
    ("sgemm_expert_plan", "offsets", None), ("sgemm_expert_plan", "rows", None), ("sgemm_expert_plan", "slots", None),
    ("sgemm_expert_linear", "top", 0), ("sgemm_expert_linear", "experts", 0), ("sgemm_expert_linear", "gather", 2),
    ("sgemm_expert_linear", "x", None), ("sgemm_expert_linear", "w", None), ("sgemm_expert_linear", "stride_w", 383),
    ("sgemm_expert_linear", "act", 9), ("sgemm_expert_linear", "offsets", None), ("sgemm_expert_linear", "rows", None),
    ("sgemm_expert_linear", "y", None), ("sgemm_expert_linear", "ldz", 1),
    ("sgemm_expert_linear_backward", "dy", None), ("sgemm_expert_linear_backward", "preact", None),
    ("sgemm_expert_linear_backward", "offsets", None), ("sgemm_expert_linear_backward", "rows", None),
    ("sgemm_expert_linear_backward", "slots", None), ("sgemm_expert_linear_backward", "lddx", 1),
    ("sgemm_expert_linear_backward", "stride_dw", 5),
    ("sgemm_expert_combine", "x", None), ("sgemm_expert_combine", "slots", None), ("sgemm_expert_combine", "ldr", 1),
    ("sgemm_expert_combine", "y", None),
    ("sgemm_expert_combine_backward", "dy", None), ("sgemm_expert_combine_backward", "x", None),
    ("sgemm_expert_combine_backward", "rows", None), ("sgemm_expert_combine_backward", "slots", None),
    ("sgemm_expert_combine_backward", "lddx", 2),
]


@pytest.mark.parametrize("name,arg,value", BAD)
def test_invalid_argument_is_named(lib, name, arg, value):
    position = NAMES[name].split().index(arg) + 1
    assert _call(lib, name, **{arg: value}) == -position
    assert "argument %d" % position in pg.last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="relies on the library failing without a device")
@pytest.mark.parametrize("name", NAMES)
def test_valid_arguments_reach_the_device_query(lib, name):
    assert _call(lib, name) == 2  # SGEMM_ERR_NO_DEVICE


def test_calls_with_nothing_to_do_touch_no_device(lib):
    assert _call(lib, "sgemm_linear", t=0, x=None, w=None, y=None) == 0
    assert _call(lib, "sgemm_linear_backward", dx=None, dw=None, dbias=None) == 0
    assert _call(lib, "sgemm_route", tokens=0, logits=None) == 0
    assert _call(lib, "sgemm_expert_linear", tokens=0, x=None) == 0
    assert _call(lib, "sgemm_expert_combine", n=0, x=None) == 0


def test_binding_refuses_host_tensors_and_bad_names():
    x, w = torch.randn(3, 4), torch.randn(5, 4)
    for call in (lambda: pg.linear(x, w), lambda: pg.linear_backward(torch.randn(3, 5), x, w),
                 lambda: pg.route(torch.randn(3, 8), 2), lambda: pg.expert_plan(torch.zeros(3, 2, dtype=torch.int32), 4),
                 lambda: pg.linear(torch.randn(4), w), lambda: pg.linear("x", w)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses_mismatched_tensors():
    x, w = torch.randn(6, 16, device="cuda"), torch.randn(24, 16, device="cuda")
    b = torch.randn(24, device="cuda")
    plan = pg.expert_plan(torch.zeros(3, 2, dtype=torch.int32, device="cuda"), 4)
    we = torch.randn(4, 24, 16, device="cuda")
    before = pg.launch_count()
    bad = [
        lambda: pg.linear(x, w[:, :15]), lambda: pg.linear(x.half(), w.half()), lambda: pg.linear(x, w.bfloat16()),
        lambda: pg.linear(x, w, b[:20]), lambda: pg.linear(x, w, b, "tanh"), lambda: pg.linear(x, w.t().contiguous().t()),
        lambda: pg.linear(x[:1].expand(6, 16), w), lambda: pg.linear(x, w, residual=torch.zeros(6, 23, device="cuda")),
        lambda: pg.linear(x, w, out=torch.zeros(6, 24)), lambda: pg.linear(x, w, b.cpu()),
        lambda: pg.linear_backward(torch.zeros(6, 24, device="cuda"), x, w, "gelu"),
        lambda: pg.linear_backward(torch.zeros(5, 24, device="cuda"), x, w),
        lambda: pg.route(x, 2, "max"), lambda: pg.route(x, 2, mask=torch.ones(6, device="cuda")),
        lambda: pg.route(x, 2, bias=torch.zeros(15, device="cuda")),
        lambda: pg.route_backward(torch.zeros(6, 2, device="cuda"), x, torch.zeros(6, 2, device="cuda")),
        lambda: pg.expert_plan(torch.zeros(3, 2, dtype=torch.int64, device="cuda"), 4),
        lambda: pg.expert_linear(x[:5], we, plan), lambda: pg.expert_linear(x[:4], we, plan, gather=True),
        lambda: pg.expert_linear(x, we[:3], plan), lambda: pg.expert_linear(x, we, "plan"),
        lambda: pg.expert_combine(x[:5], plan), lambda: pg.expert_combine(x, plan, torch.zeros(3, 1, device="cuda")),
        lambda: pg.expert_combine_backward(x, x, plan),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pg.SgemmError):
        pg.route(x, 17)
    assert pg.launch_count() == before
