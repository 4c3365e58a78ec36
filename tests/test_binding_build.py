"""The C library and the Python binding of the short calls are built and loaded apart: what needs only the library does
not need torch's headers, a host compiler or the binding."""

import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

from blockwise_exact_attention_gb300 import _lib, build  # noqa: E402
import blockwise_exact_attention_gb300 as bea  # noqa: E402


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small source in a folder of its own."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libbea.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / os.path.basename(build.BIND)))
    monkeypatch.setattr(build, "_sources", lambda: [os.path.join(build.CSRC, "selftest.cu")])
    return tmp_path


def no_torch():
    raise ModuleNotFoundError("No module named 'torch'")


def no_compiler():
    return ["a-compiler-that-does-not-exist"]


@pytest.mark.parametrize("name,broken", [("_torch_paths", no_torch), ("_host_compiler", no_compiler)])
def test_the_library_is_built_without_the_binding(elsewhere, monkeypatch, capfd, name, broken):
    monkeypatch.setattr(build, name, broken)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BIND)
    assert "binding" in capfd.readouterr().err                     # said, not hidden
    at = os.stat(build.LIB).st_mtime_ns
    assert build.build() == build.LIB and os.stat(build.LIB).st_mtime_ns == at   # the library stays, the binding is tried again
    assert "binding" in capfd.readouterr().err


def test_a_failed_binding_leaves_no_older_one(elsewhere, monkeypatch):
    with open(build.BIND, "w") as f:
        f.write("of an earlier build")
    monkeypatch.setattr(build, "_torch_paths", no_torch)
    build.build(force=True)
    assert not os.path.exists(build.BIND)


def test_an_error_in_the_library_is_raised(elsewhere, monkeypatch):
    bad = elsewhere / "bad.cu"
    bad.write_text("not C++")
    monkeypatch.setattr(build, "_sources", lambda: [str(bad)])
    monkeypatch.setattr(build, "_torch_paths", no_torch)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()


def test_launches_are_counted_without_the_binding(monkeypatch):
    def fail():
        raise RuntimeError("no binding here")
    monkeypatch.setattr(_lib, "_BIND", None)
    monkeypatch.setattr(_lib, "bind", fail)
    monkeypatch.setattr(bea.ops, "_launches", 3)
    assert bea.launches_since_reset() == 3 and bea.launches_since_reset(reset=True) == 3
    assert bea.launches_since_reset() == 0


def test_launches_are_counted_before_anything_is_loaded():
    """As before the binding was there: a count asks for no library."""
    code = ("import blockwise_exact_attention_gb300 as bea, blockwise_exact_attention_gb300._lib as l\n"
            "print(bea.launches_since_reset(reset=True), l._LIB, l._BIND)")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build.ROOT, timeout=300)
    assert r.stdout.split() == ["0", "None", "None"], r.stderr[-2000:]


def test_a_missing_binding_is_an_error_that_names_it(monkeypatch, tmp_path):
    build.build()
    _lib.load()
    monkeypatch.setattr(_lib, "_BIND", None)
    monkeypatch.setattr(build, "BIND", str(tmp_path / "_bind.so"))
    with pytest.raises(RuntimeError, match="binding"):
        _lib.bind()


def test_a_binding_of_another_torch_or_python_is_built_anew(monkeypatch):
    import sysconfig
    import torch
    build.build()
    assert build.binding_up_to_date() and build.up_to_date()
    of = build.binding_stamp()
    assert torch.__version__ in of and sysconfig.get_config_var("SOABI") in of
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0")
        assert not build.binding_up_to_date() and not build.up_to_date() and build.library_up_to_date()
    with monkeypatch.context() as m:
        m.setattr(build, "BINDING_FLAGS", ["-O0"])
        assert not build.binding_up_to_date()
    assert build.binding_up_to_date()


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    import torch
    build.build()
    monkeypatch.setattr(_lib, "_BIND", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0")
        with pytest.raises(RuntimeError, match="1.0.0"):
            _lib.bind()
    _lib.bind()


def test_the_binding_needs_no_intermediate_files(monkeypatch, tmp_path):
    """Neither the objects nor the log of its build."""
    build.build()
    monkeypatch.setattr(_lib, "_BIND", None)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "cleaned"))
    assert build.up_to_date()
    _lib.bind()
