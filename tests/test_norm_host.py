"""Refusals of the layer norm calls that need no GPU: the library names the first invalid
argument before it touches a device, and the binding refuses tensors it cannot pass."""
import pytest
import torch

import precision_gemm_gb300 as pg
from precision_gemm_gb300 import build as pgbuild

P = 4096  # an address that is never dereferenced
NAMES = {
    "sgemm_layer_norm": "dtype t n x ldx w bias eps y ldy mean rstd stream",
    "sgemm_layer_norm_backward": "dtype t n dy lddy x ldx w mean rstd residual ldr dx lddx dw dbias stream",
}
GOOD = dict(dtype=1, t=4, n=24, ldx=24, eps=1e-5, ldy=24, lddy=24, ldr=24, lddx=24, stream=None)


@pytest.fixture(scope="module")
def lib():
    pgbuild.build()
    return pg.load_library()


def _call(lib, name, **bad):
    args = {**GOOD, **bad}
    return getattr(lib, name)(*[args.get(a, P) for a in NAMES[name].split()])


BAD = [("sgemm_layer_norm", "dtype", 2), ("sgemm_layer_norm", "t", -1), ("sgemm_layer_norm", "t", 2 ** 31),
       ("sgemm_layer_norm", "n", 0), ("sgemm_layer_norm", "x", None), ("sgemm_layer_norm", "ldx", 23),
       ("sgemm_layer_norm", "eps", -1e-9), ("sgemm_layer_norm", "eps", float("nan")),
       ("sgemm_layer_norm", "eps", float("inf")), ("sgemm_layer_norm", "y", None), ("sgemm_layer_norm", "ldy", 0)]
BAD += [("sgemm_layer_norm_backward", a, v) for a, v in (
    ("dtype", -1), ("n", 0), ("dy", None), ("lddy", 1), ("x", None), ("ldx", 1), ("mean", None), ("rstd", None),
    ("ldr", 23), ("lddx", 23))]


@pytest.mark.parametrize("name,arg,value", BAD)
def test_invalid_argument_is_named(lib, name, arg, value):
    position = NAMES[name].split().index(arg) + 1
    assert _call(lib, name, **{arg: value}) == -position
    assert "argument %d" % position in pg.last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="relies on the library failing without a device")
@pytest.mark.parametrize("name", NAMES)
def test_valid_arguments_reach_the_device_query(lib, name):
    assert _call(lib, name) == 2  # SGEMM_ERR_NO_DEVICE
    optional = {"sgemm_layer_norm": dict(w=None, bias=None, mean=None, rstd=None),
                "sgemm_layer_norm_backward": dict(w=None, residual=None, ldr=0, dw=None)}
    assert _call(lib, name, **optional[name]) == 2


def test_calls_with_nothing_to_do_touch_no_device(lib):
    assert _call(lib, "sgemm_layer_norm", t=0, x=None, y=None) == 0
    assert _call(lib, "sgemm_layer_norm_backward", dx=None, dw=None, dbias=None, dy=None, mean=None) == 0
    assert _call(lib, "sgemm_layer_norm_backward", t=0, dw=None, dbias=None, dy=None, mean=None) == 0


def test_binding_refuses_host_tensors():
    x = torch.randn(3, 4)
    for call in (lambda: pg.layer_norm(x), lambda: pg.layer_norm("x"), lambda: pg.layer_norm(x[0]),
                 lambda: pg.layer_norm_backward(x, x, None, x[:, 0], x[:, 0])):
        with pytest.raises(ValueError):
            call()
