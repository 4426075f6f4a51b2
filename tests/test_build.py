"""The build: the C library without the Python binding, and a binding for another torch."""
import os

import pytest

import torch

from mbarrier_async_tile_gb300 import _build, layer


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The binding, its object and its stamp in a folder of their own."""
    _build.build()
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "BINDING_PATH", str(tmp_path / "binding.so"))
    monkeypatch.setattr(_build, "BINDING_STAMP", str(tmp_path / "binding.stamp"))
    monkeypatch.setattr(_build, "binding_error", None)
    monkeypatch.setattr(layer, "_compiled", None)
    return tmp_path


def without_headers():
    raise RuntimeError("no headers here")


def test_library_is_built_where_the_binding_cannot_be(elsewhere, monkeypatch):
    monkeypatch.setattr(_build, "_binding_flags", without_headers)
    monkeypatch.setattr(_build, "SOURCES", ["mbtile_probe.cu"])          # (one quick unit, linked aside)
    monkeypatch.setattr(_build, "LIB_PATH", str(elsewhere / "libmbtile.so"))
    (elsewhere / "binding.so").write_text("of another time")
    with pytest.warns(UserWarning, match="no headers here"):
        assert _build.build() == str(elsewhere / "libmbtile.so")
    assert os.path.getsize(elsewhere / "libmbtile.so") > 0
    assert not (elsewhere / "binding.so").exists()
    assert _build.build() == str(elsewhere / "libmbtile.so")             # not tried again, nor warned of
    with pytest.raises(RuntimeError, match="no headers here"):
        layer._ext()


def test_binding_of_another_torch_is_built_anew(elsewhere, monkeypatch):
    made = []
    monkeypatch.setattr(_build, "_compile_binding", lambda: "object")
    monkeypatch.setattr(_build, "_run", lambda cmd, what: made.append(what) or (elsewhere / cmd[3]).write_text("x") and "")
    _build.build()
    _build.build()
    assert made == ["link of the binding"]
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    _build.build()
    _build.build()
    assert made == ["link of the binding"] * 2
