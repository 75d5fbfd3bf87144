"""The bindings in C of the serving operators, called as a module."""
import os
import re

import pytest

from gemv_mul_mm_gb300 import build as qbuild
from gemv_mul_mm_gb300 import qmm

SOURCE = os.path.join(os.path.dirname(qbuild.__file__), "csrc", "pycall.c")


@pytest.fixture(scope="module")
def M():
    qbuild.build()
    return qmm._calls()


@pytest.mark.parametrize("name,n", [("qrope", 7), ("qkv_store", 12), ("qkv_load", 9), ("qattn_decode", 16)])
def test_argument_counts(M, name, n):
    for k in {0, 1, n - 1, n + 1}:
        with pytest.raises(TypeError):
            getattr(M, name)(*[None] * k)


def test_no_argument_is_read_before_they_are_counted():
    """Reading args[i] of a shorter call reads past the caller's array."""
    text = open(SOURCE).read()
    bodies = re.findall(r"PyObject \*const \*a, Py_ssize_t n\) \{(.*?)\n\}", text, re.S)
    assert len(bodies) == 4
    for body in bodies:
        assert re.search(r"\ba\[", body).start() > body.index("nargs_are(n,")


@pytest.mark.gpu
def test_tables_longer_than_an_int_are_refused(M):
    """2 * numel of a turns table is an int of the call: 2^31 + 32 entries are not 32."""
    import torch
    x = torch.zeros((1, 1, 64), device="cuda")
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        qmm.qrope(x, pos, torch.empty((1 << 31) + 32, dtype=torch.int64, device="cuda"))
