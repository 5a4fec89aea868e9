"""What the build makes, with small sources in a folder of their own."""
import os
import sys
import warnings

import pytest
import torch

import positional_lsh_approximation_gb300 as plsh

build_mod = plsh._build_mod


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source folder of one unit and a binding that needs no headers."""
    src, out = tmp_path / "csrc", tmp_path / "_build"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (src / "binding.cpp").write_text('extern "C" int two() { return 2; }\n')
    monkeypatch.setattr(build_mod, "SRC_DIR", str(src))
    monkeypatch.setattr(build_mod, "BUILD_DIR", str(out))
    monkeypatch.setattr(build_mod, "LIB_PATH", str(out / "libplsh.so"))
    monkeypatch.setattr(build_mod, "BINDING_PATH", str(out / "_plsh_binding.so"))
    monkeypatch.setattr(build_mod, "SOURCES", ["one.cu"])
    return src


def test_library_and_binding_are_built_once(tree):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert build_mod.build() == build_mod.LIB_PATH
        made = [os.stat(p).st_mtime_ns for p in (build_mod.LIB_PATH, build_mod.BINDING_PATH)]
        build_mod.build()
    assert made == [os.stat(p).st_mtime_ns for p in (build_mod.LIB_PATH, build_mod.BINDING_PATH)]


def test_the_library_does_not_need_the_binding(tree, monkeypatch):
    """A box without torch's or Python's headers gets the C library, and the
    calls that go through the binding say what is missing."""
    build_mod.build()
    os.remove(build_mod.LIB_PATH)
    (tree / "binding.cpp").write_text("#error headers are missing here\n")
    os.utime(tree / "binding.cpp", (2 ** 31, 2 ** 31))
    with pytest.warns(RuntimeWarning, match="headers are missing here"):
        build_mod.build()
    assert os.path.exists(build_mod.LIB_PATH)
    assert not os.path.exists(build_mod.BINDING_PATH)          # nor one of other sources
    monkeypatch.setattr(plsh, "_native", None)
    monkeypatch.setattr(plsh, "load", lambda: None)
    with pytest.raises(RuntimeError, match="binding"):
        plsh._binding()


def test_the_library_does_not_need_a_host_compiler_for_the_binding(tree, monkeypatch):
    monkeypatch.setattr(build_mod, "_binding_compile", lambda out: [os.path.join(str(tree), "no-such-compiler")])
    with pytest.warns(RuntimeWarning, match="no-such-compiler"):
        build_mod.build()
    assert os.path.exists(build_mod.LIB_PATH)


def test_the_library_does_not_need_torch(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)            # import torch raises
    with pytest.warns(RuntimeWarning, match="torch"):
        build_mod.build()
    assert os.path.exists(build_mod.LIB_PATH)


def test_a_binding_of_another_torch_is_not_used(tree, monkeypatch):
    build_mod.build()
    made = os.stat(build_mod.BINDING_PATH).st_mtime_ns
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    # without a build: refused before it is loaded
    monkeypatch.setattr(plsh, "_native", None)
    monkeypatch.setattr(plsh, "load", lambda: None)
    with pytest.raises(RuntimeError, match="0.0.0"):
        plsh._binding()
    # a build makes it anew, once, and leaves the library
    lib = os.stat(build_mod.LIB_PATH).st_mtime_ns
    build_mod.build()
    anew = os.stat(build_mod.BINDING_PATH).st_mtime_ns
    assert anew != made and os.stat(build_mod.LIB_PATH).st_mtime_ns == lib
    build_mod.build()
    assert os.stat(build_mod.BINDING_PATH).st_mtime_ns == anew


def test_a_unit_that_does_not_compile_is_an_error(tree):
    (tree / "one.cu").write_text("#error not this one\n")
    with pytest.raises(RuntimeError):
        build_mod.build()
