"""The compiled module of the layer operators' calls: which file it is, and
what happens without it."""

import os
import sysconfig

import pytest
import torch

import latent_projection_top_gb300 as route
from latent_projection_top_gb300 import builder, layer


@pytest.fixture(scope="module", autouse=True)
def _built():
    route.build()


def test_module_is_this_torch_and_this_python():
    """Built for another torch or Python it would read tensors through the
    wrong layout: each has a file of its own."""
    name = os.path.basename(builder.call_module())
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name
    assert os.path.exists(builder.call_module())
    layer._short_way()


def test_another_torch_is_another_module(tmp_path, monkeypatch):
    here = builder.call_module()
    (tmp_path / "version.py").write_text("__version__ = '9.9.9+cu999'\n")
    monkeypatch.setattr(builder, "_torch_dir", lambda: str(tmp_path))
    other = builder.call_module()
    assert other != here and "9.9.9+cu999" in other
    assert builder._stale(other, [builder.CALL_SOURCE])


def test_build_without_torch_or_its_headers(tmp_path, monkeypatch):
    """The library does not need the module: build() goes on, and says so."""
    monkeypatch.setattr(builder, "_torch_dir", lambda: None)
    with pytest.warns(UserWarning, match="torch is not installed"):
        assert builder.build() == builder.LIB
    (tmp_path / "version.py").write_text("__version__ = '9.9.9'\n")  # and no include/
    monkeypatch.setattr(builder, "_torch_dir", lambda: str(tmp_path))
    with pytest.warns(UserWarning, match="layer_call.cpp"):
        assert builder.build() == builder.LIB
    assert not os.path.exists(builder.call_module())


def test_binding_without_the_module(tmp_path, monkeypatch):
    monkeypatch.setattr(layer, "_short", None)
    monkeypatch.setattr(layer, "_without", False)
    for path in (tmp_path / "missing.so", tmp_path / "broken.so"):
        if path.name == "broken.so":
            path.write_bytes(b"not a library")
        monkeypatch.setattr(layer, "_without", False)
        monkeypatch.setattr(builder, "call_module", lambda p=path: str(p))
        with pytest.warns(UserWarning, match="ctypes"):
            assert layer._short_way() is None
        assert layer._short_way() is None  # warned once
