"""Refusals of the gated linear calls that need no GPU: the library names the first invalid
argument before it touches a device, and the binding refuses tensors it cannot pass."""
import pytest
import torch

import precision_gemm_gb300 as pg
from precision_gemm_gb300 import build as pgbuild

P = 4096  # an address that is never dereferenced
NAMES = {
    "sgemm_gated_linear": "dtype t n k x ldx w ldw bias act y ldy preact ldz stream",
    "sgemm_gated_linear_backward": "dtype t n k dy lddy x ldx w ldw act preact ldz dx lddx dw lddw dbias stream",
}
GOOD = dict(dtype=1, t=4, n=24, k=16, ldx=16, ldw=16, act=2, ldy=24, ldz=48, lddy=24, lddx=16, lddw=16, stream=None)


@pytest.fixture(scope="module")
def lib():
    pgbuild.build()
    return pg.load_library()


def _call(lib, name, **bad):
    args = {**GOOD, **bad}
    return getattr(lib, name)(*[args.get(a, P) for a in NAMES[name].split()])


BAD = [("sgemm_gated_linear", a, v) for a, v in (
    ("dtype", 2), ("t", -1), ("n", 2 ** 30), ("k", 2 ** 31), ("x", None), ("ldx", 15), ("w", None), ("ldw", 15),
    ("act", 5), ("y", None), ("ldy", 23), ("ldz", 47))]
BAD += [("sgemm_gated_linear_backward", a, v) for a, v in (
    ("dtype", -1), ("n", 2 ** 30), ("dy", None), ("lddy", 23), ("x", None), ("w", None), ("act", -1), ("preact", None),
    ("ldz", 47), ("lddx", 15), ("lddw", 15))]


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
    assert _call(lib, "sgemm_gated_linear", t=0, x=None, w=None, y=None) == 0
    assert _call(lib, "sgemm_gated_linear", n=0, x=None, w=None, y=None) == 0
    assert _call(lib, "sgemm_gated_linear_backward", dx=None, dw=None, dbias=None, dy=None, preact=None) == 0


def test_binding_refuses_host_tensors():
    x, w = torch.randn(3, 4), torch.randn(10, 4)
    for call in (lambda: pg.gated_linear(x, w), lambda: pg.gated_linear(x[0], w), lambda: pg.gated_linear("x", w),
                 lambda: pg.gated_linear_backward(torch.randn(3, 5), x, w, torch.randn(3, 10))):
        with pytest.raises(ValueError):
            call()
