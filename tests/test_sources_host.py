"""What the CUDA sources may not use, read as text: no GPU and no build needed."""
import os
import re

import pytest

from precision_gemm_gb300 import build as pgbuild

SOURCES = [os.path.join(pgbuild.CSRC, f) for f in sorted(os.listdir(pgbuild.CSRC))]


def _code(path):
    """The source without its comments, adjacent string literals joined."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r'"\s*"', "", text)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_bulk_load_is_multicast(path):
    """The library serves programs of several GPUs too, where a tensor map may cover another GPU's
    memory: every bulk copy goes to one thread block's shared memory."""
    for statement in re.findall(r"cp\.async\.bulk[^;]*;", _code(path)):
        assert "multicast" not in statement, statement


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_takes_its_data_for_constant(path):
    """Kernels start while the one before them still writes what they read (programmatic launches), and
    wait for it inside: a non-coherent load is for data that is constant while its kernel runs."""
    code = _code(path)
    assert "ld.global.nc" not in code and not re.search(r"\b__ldg\s*\(", code)
