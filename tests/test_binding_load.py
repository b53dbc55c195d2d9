"""Which compiled module the package loads (no GPU), and that it goes on without one."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

from conftest import ROOT

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def built():
    import torch
    from __graft_entry__ import _build_module, build
    build()
    return os.path.join(ROOT, "paged_kv_cache_261_gb300"), os.path.basename(_build_module().binding_path(torch.__version__))


def package(built, tmp_path):
    """A copy of the package that shares the library, without a module."""
    folder, _ = built
    copy = tmp_path / "paged_kv_cache_261_gb300"
    os.makedirs(copy / "_build")
    for f in os.listdir(folder):
        if f.endswith(".py"):
            shutil.copy(os.path.join(folder, f), copy)
    os.symlink(os.path.join(folder, "_build", "libpagedattn.so"), copy / "_build" / "libpagedattn.so")
    return copy


def state_of(tmp_path):
    """What the copy says of its module after its first use of torch, and the warnings."""
    code = ("import sys, warnings; sys.path.insert(0, sys.argv[1])\n"
            "with warnings.catch_warnings(record=True) as w:\n"
            "    warnings.simplefilter('always')\n"
            "    import paged_kv_cache_261_gb300 as pa\n"
            "    import torch\n"
            "    try:\n"
            "        pa.paged_kv_write_fp8_block(*[torch.zeros(1)] * 6)\n"
            "    except ValueError as e:\n"
            "        print(e)\n"
            "print(pa._binding is not None, [str(x.message) for x in w if 'ctypes' in str(x.message)])")
    r = subprocess.run([sys.executable, "-c", code, str(tmp_path)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    said, last = r.stdout.strip().split("\n")[-2:]
    assert "must be a CUDA tensor" in said
    return last


def test_a_module_that_cannot_be_imported(built, tmp_path):
    """Not a shared object, or built for something else: a warning, and the calls go the Python code's way."""
    copy = package(built, tmp_path)
    (copy / "_build" / built[1]).write_text("no module")
    last = state_of(tmp_path)
    assert last.startswith("False") and built[1] in last


def test_no_module(built, tmp_path):
    package(built, tmp_path)
    assert state_of(tmp_path) == "False []"


def test_module_of_another_python(built, tmp_path):
    """The interpreter's tag is part of the name, so a module of another one is not looked at."""
    tag = sysconfig.get_config_var("SOABI")
    assert tag in built[1]
    copy = package(built, tmp_path)
    (copy / "_build" / built[1].replace(tag, "cpython-399-other")).write_text("no module")
    assert state_of(tmp_path) == "False []"


FAKE = """
#include <Python.h>
static PyObject *interface(PyObject *self, PyObject *args) { return Py_BuildValue("KKK", 1ull, %s, 0ull); }
static PyMethodDef methods[] = {{"%s", interface, METH_NOARGS, NULL}, {NULL, NULL, 0, NULL}};
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pagedattn_binding", NULL, -1, methods};
PyMODINIT_FUNC PyInit__pagedattn_binding(void) { return PyModule_Create(&module); }
"""


@pytest.mark.parametrize("library,name", [("2ull", "interface"), ("1ull", "interface"), ("1ull", "something_else")])
def test_a_module_of_another_library(built, tmp_path, library, name):
    """Built with another header than the library, calling another copy of it, or from before modules said so."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        pytest.skip("no Python.h")
    copy = package(built, tmp_path)
    (tmp_path / "fake.c").write_text(FAKE % (library, name))
    subprocess.run(["gcc", "-shared", "-fPIC", "-I" + include, str(tmp_path / "fake.c"), "-o", str(copy / "_build" / built[1])],
                   check=True)
    last = state_of(tmp_path)
    assert last.startswith("False") and built[1] in last


def test_the_module_that_was_built(built, tmp_path):
    """It is taken, and says the header's number."""
    from __graft_entry__ import _build_module
    if not os.path.exists(os.path.join(built[0], "_build", built[1])):
        pytest.skip("no compiled module here")
    copy = package(built, tmp_path)
    os.symlink(os.path.join(built[0], "_build", built[1]), copy / "_build" / built[1])
    assert state_of(tmp_path) == "True []"
    import paged_kv_cache_261_gb300 as pa
    pa._torch()
    compiled, library, _ = pa._binding.interface()
    assert compiled == library == int(_build_module().interface().split("=")[1][:-3], 16)
