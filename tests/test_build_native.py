"""CPU test of the build where the interpreter's headers are not installed."""
import sysconfig

import pytest

import structured_mask_linear_gb300 as sml
from structured_mask_linear_gb300 import _build


def test_without_python_headers(tmp_path, monkeypatch):
    """The C library is built all the same; the calls that need the CPython module say what is
    missing."""
    _build.build()
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda: paths)
    monkeypatch.setattr(_build, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(sml, "_NATIVE_PATH", str(tmp_path / "_native.so"))
    monkeypatch.setattr(sml, "_native_module", None)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert _build.build() == _build.LIB
    with pytest.raises(RuntimeError, match="Python.h"):
        sml.lindecay_fwd(None, None, None, None)
    assert sml.loglinear_status_string(0) == "ok"
