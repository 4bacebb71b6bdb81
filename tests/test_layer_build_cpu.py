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
