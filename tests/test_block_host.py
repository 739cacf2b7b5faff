"""Refusals of the 8-bit matrix calls that need no GPU: the library names the first invalid
argument before it touches a device, and the binding refuses tensors it cannot pass."""
import pytest
import torch

import precision_gemm_gb300 as pg
from precision_gemm_gb300 import build as pgbuild

P = 4096  # an address that is never dereferenced
NAMES = {
    "sgemm_quantize": "dtype t k block_rows x ldx q ldq scales lds stream",
    "sgemm_block_linear": "dtype t n k x ldx x_scales ldxs w ldw w_scales ldws bias act residual ldr y ldy stream",
}
GOOD = dict(dtype=1, t=4, n=24, k=200, block_rows=1, ldx=200, ldq=200, lds=2, ldxs=2, ldw=200, ldws=2, act=2, ldr=24,
            ldy=24, stream=None)


@pytest.fixture(scope="module")
def lib():
    pgbuild.build()
    return pg.load_library()


def _call(lib, name, **bad):
    args = {**GOOD, **bad}
    return getattr(lib, name)(*[args.get(a, P) for a in NAMES[name].split()])


BAD = [("sgemm_quantize", a, v) for a, v in (
    ("dtype", 2), ("t", -1), ("k", 2 ** 31), ("block_rows", 64), ("block_rows", 0), ("x", None), ("ldx", 199),
    ("q", None), ("ldq", 199), ("scales", None), ("lds", 1))]
BAD += [("sgemm_block_linear", a, v) for a, v in (
    ("dtype", -1), ("t", -1), ("n", 2 ** 31), ("k", -1), ("x", None), ("ldx", 199), ("ldxs", 1), ("w", None),
    ("ldw", 199), ("w_scales", None), ("ldws", 1), ("act", 5), ("ldr", 23), ("y", None), ("ldy", 23))]


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
    assert _call(lib, "sgemm_quantize", t=0, x=None, q=None, scales=None) == 0
    assert _call(lib, "sgemm_quantize", k=0, x=None, q=None, scales=None) == 0
    assert _call(lib, "sgemm_block_linear", t=0, x=None, w=None, w_scales=None, y=None) == 0


def test_binding_refuses_host_tensors():
    x, w = torch.randn(3, 4), torch.zeros(5, 4, dtype=torch.float8_e4m3fn)
    for call in (lambda: pg.quantize(x), lambda: pg.quantize("x"), lambda: pg.block_linear(x, w, torch.ones(1, 1)),
                 lambda: pg.block_linear(w, w, torch.ones(1, 1), x_scales=torch.ones(5, 1))):
        with pytest.raises(ValueError):
            call()
