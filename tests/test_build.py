"""The build of the library and of the compiled module beside it (no GPU): the package does not depend on the module."""
import importlib.util
import os
import subprocess
import sys

import pytest

from conftest import ROOT


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build script with a folder of its own and a library of its smallest source."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "paged_kv_cache_261_gb300", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(m, "BUILD", str(tmp_path))
    monkeypatch.setattr(m, "LIB", str(tmp_path / "libpagedattn.so"))
    monkeypatch.setattr(m, "SOURCES", ["allocator.cpp"])
    return m


def counted(monkeypatch, build):
    """The commands that the build runs."""
    seen, inner = [], build._run
    monkeypatch.setattr(build, "_run", lambda cmd, what: (seen.append(what), inner(cmd, what))[1])
    return seen


@pytest.mark.parametrize("broken", ["the command", "the compilation", "the link"])
def test_library_without_its_module(monkeypatch, build, broken):
    """No Python.h, no CUDA headers for torch's, no torch libraries: the library is built all the same, with a
    warning; the module is not tried again until a source changes."""
    pytest.importorskip("torch")

    def no_headers(obj):
        raise RuntimeError("no headers")

    if broken == "the command":
        monkeypatch.setattr(build, "_binding_command", no_headers)
    elif broken == "the compilation":
        monkeypatch.setattr(build, "_binding_command", lambda obj: ["g++", "-c", os.path.join(ROOT, "README.md.cpp"), "-o", obj])
    else:
        monkeypatch.setattr(build, "_binding_command", lambda obj: ["g++", "-x", "c++", "-c", os.devnull, "-o", obj])
        monkeypatch.setattr(build, "_link_binding", lambda *a: build._run(["g++", "-lno_such_library"], "linking the binding"))
    seen = counted(monkeypatch, build)
    with pytest.warns(UserWarning, match="compiled module"):
        assert build.build_library() == build.LIB
    assert os.path.exists(build.LIB) and "compiling allocator.cpp" in seen
    left = sorted(os.listdir(build.BUILD))
    assert [f for f in left if f.endswith(".so")] == ["libpagedattn.so"] and not [f for f in left if f.endswith(".o")]
    del seen[:]
    build.build_library()
    assert not seen
    os.utime(os.path.join(build.BUILD, next(f for f in left if f.endswith(".failed"))), (1, 1))   # older than the sources
    with pytest.warns(UserWarning, match="compiled module"):
        build.build_library()
    assert "compiling allocator.cpp" not in seen


def test_library_that_does_not_compile_is_an_error(monkeypatch, build):
    monkeypatch.setattr(build, "SOURCES", ["allocator.cpp", "no_such_source.cu"])
    monkeypatch.setattr(build, "_torch_version", lambda: None)
    with pytest.raises(RuntimeError, match="no_such_source"):
        build.build_library()
    assert not os.path.exists(build.LIB)


def test_looking_for_something_to_build_does_not_import_torch():
    pytest.importorskip("torch")
    code = ("import importlib.util, sys; s = importlib.util.spec_from_file_location('b', sys.argv[1]); "
            "m = importlib.util.module_from_spec(s); s.loader.exec_module(m); "
            "m._stale = lambda path: False; m.build_library(); assert 'torch' not in sys.modules; print(m._torch_version())")
    r = subprocess.run([sys.executable, "-c", code, os.path.join(ROOT, "paged_kv_cache_261_gb300", "build.py")],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    import torch
    assert r.stdout.strip() == (torch.__version__ if torch.version.cuda else "None")


@pytest.mark.parametrize("links", [True, False])
def test_a_new_library_leaves_no_old_module_beside_it(monkeypatch, build, links):
    """The module is linked before the library is replaced; those of the old one, for any torch, are gone."""
    torch = pytest.importorskip("torch")
    for f in (build.binding_path("1.0"), build.binding_path(torch.__version__), build.binding_path("1.0") + ".failed", build.LIB):
        with open(f, "w") as h:
            h.write("old")
    monkeypatch.setattr(build, "_binding_command", lambda obj: ["g++", "-x", "c++", "-c", os.devnull, "-o", obj])

    def link(obj, folder, to):
        with open(build.LIB) as h:
            assert h.read() == "old"
        assert os.path.getsize(os.path.join(folder, "libpagedattn.so")) > 1000
        if not links:
            raise RuntimeError("does not link")
        with open(to, "w") as h:
            h.write("new")

    monkeypatch.setattr(build, "_link_binding", link)
    if links:
        build.build_library(force=True)
    else:
        with pytest.warns(UserWarning, match="does not link"):
            build.build_library(force=True)
    path = build.binding_path(torch.__version__)
    assert sorted(os.listdir(build.BUILD)) == sorted([os.path.basename(path) + ("" if links else ".failed"), "libpagedattn.so"])
    assert os.path.getsize(build.LIB) > 1000


def test_the_interface_is_the_header(monkeypatch, build, tmp_path):
    a = build.interface()
    other = tmp_path / "pagedattn.h"
    other.write_text(open(build.HEADER).read() + "int pa_one_more(void);\n")
    monkeypatch.setattr(build, "HEADER", str(other))
    assert a.startswith("-DPA_INTERFACE=0x") and a.endswith("ull") and build.interface() != a
