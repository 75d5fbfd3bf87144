"""gemv_mul_mm_gb300/build.py: the library does not depend on what the Python
bindings need, and these are named for the Python that they are built for."""
import os
import sysconfig

import pytest

from gemv_mul_mm_gb300 import build as qbuild


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The bindings go to a folder of the test; returns it."""
    qbuild.build()
    monkeypatch.setattr(qbuild, "PYCALL", str(tmp_path / os.path.basename(qbuild.PYCALL)))
    return tmp_path


def test_library_without_python_headers(elsewhere, monkeypatch, capsys):
    paths = dict(sysconfig.get_paths(), include=str(elsewhere / "no_headers_here"))
    monkeypatch.setattr(qbuild.sysconfig, "get_paths", lambda *a, **kw: paths)
    assert qbuild.build() == qbuild.LIB and os.path.exists(qbuild.LIB)
    assert os.listdir(elsewhere) == []
    assert "Python.h" in capsys.readouterr().err


def test_library_without_a_c_compiler(elsewhere, monkeypatch, capsys):
    monkeypatch.setattr(qbuild.shutil, "which", lambda name: None)
    monkeypatch.delenv("CC", raising=False)
    assert qbuild.build() == qbuild.LIB
    assert os.listdir(elsewhere) == []
    assert "C compiler" in capsys.readouterr().err


def test_errors_in_the_bindings_are_not_hidden(elsewhere, monkeypatch):
    bad = elsewhere / "bad.c"
    bad.write_text("#error no\n")
    monkeypatch.setattr(qbuild, "PYCALL_SRC", str(bad))
    with pytest.raises(RuntimeError):
        qbuild.build()


def test_bindings_are_named_for_this_python(elsewhere):
    qbuild.build()
    assert os.listdir(elsewhere) == ["_pycall" + sysconfig.get_config_var("EXT_SUFFIX")]


def test_calls_without_the_bindings_say_so(monkeypatch):
    import sys

    from gemv_mul_mm_gb300 import qmm
    pytest.importorskip("torch")
    import gemv_mul_mm_gb300 as package
    qbuild.build()
    monkeypatch.setattr(qmm, "_CALL", None)
    monkeypatch.delattr(package, "_pycall", raising=False)
    monkeypatch.setitem(sys.modules, "gemv_mul_mm_gb300._pycall", None)
    with pytest.raises(ImportError, match="_pycall"):
        qmm.qkv_store("f16", None, None, None, None, None, 16)
