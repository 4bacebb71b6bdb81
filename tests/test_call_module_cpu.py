"""A compiled calls' module that is not this binding's: the calls go through ctypes."""

import os
import subprocess
import sysconfig

import pytest

import latent_projection_top_gb300 as route
from latent_projection_top_gb300 import builder, layer

OTHER = r"""
#include <Python.h>
static PyObject *bind(PyObject *self, PyObject *args) {
    (void)self;
    if (PyTuple_GET_SIZE(args) != TAKES) return PyErr_Format(PyExc_TypeError, "takes %d addresses", TAKES);
    Py_RETURN_NONE;
}
static PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, NULL}, {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_call", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit__layer_call(void) { return PyModule_Create(&module); }
"""


@pytest.mark.parametrize("takes", [6, 5])  # the layer operators' entry points alone; not even those
def test_a_module_of_another_version_is_not_used(tmp_path, monkeypatch, takes):
    route.build()
    source, so = tmp_path / "other.c", tmp_path / "_layer_call.so"
    source.write_text(OTHER)
    subprocess.run(["gcc", "-shared", "-fPIC", f"-DTAKES={takes}", "-I", sysconfig.get_paths()["include"],
                    str(source), "-o", str(so)], check=True)
    monkeypatch.setattr(layer, "_short", None)
    monkeypatch.setattr(layer, "_without", False)
    monkeypatch.setattr(builder, "call_module", lambda: str(so))
    with pytest.warns(UserWarning, match="ctypes"):
        assert layer._short_way() is None
    assert layer._short is None
    assert layer._short_way() is None  # warned once


def failing(*_):
    raise RuntimeError("no compiler")


def test_a_module_that_could_not_be_rebuilt_is_not_left(tmp_path, monkeypatch):
    """What build() warns of holds: a module older than its source is not loaded."""
    so = tmp_path / "_layer_call.so"
    so.write_bytes(b"")
    os.utime(so, (0, 0))
    monkeypatch.setattr(builder, "call_module", lambda: str(so))
    monkeypatch.setattr(builder, "_compile_call_module", failing)
    with pytest.warns(UserWarning, match="ctypes.*no compiler"):
        builder._build_call_module(False)
    assert not so.exists()


def test_a_module_that_is_up_to_date_stays(tmp_path, monkeypatch):
    so = tmp_path / "_layer_call.so"
    so.write_bytes(b"")
    monkeypatch.setattr(builder, "call_module", lambda: str(so))
    monkeypatch.setattr(builder, "_compile_call_module", failing)
    builder._build_call_module(False)
    assert so.exists()
    with pytest.warns(UserWarning, match="no compiler"):
        builder._build_call_module(True)
    assert so.exists()
