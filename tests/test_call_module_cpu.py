"""A compiled calls' module that is not this binding's: the calls go through ctypes."""

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
