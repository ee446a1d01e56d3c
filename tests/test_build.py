"""The build where the compiled host calls cannot be made: libpa.so stands alone."""

import ctypes
import importlib.metadata
import os
import types
import warnings

import pytest

from paged_kv_cache_254_gb300 import _build, _lib, ops


@pytest.fixture
def small_build(monkeypatch, tmp_path):
    """The build with one small source, in a folder of its own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int pa_one() { return 1; }\n')
    monkeypatch.setattr(_build, "_sources", lambda: [str(src)])
    monkeypatch.setattr(_build, "_deps", lambda: [str(src)])
    for name, file in (("LIBDIR", "lib"), ("OBJDIR", "lib/obj"), ("LIBPATH", "lib/libpa.so"), ("FASTPATH", "lib/_pa_fast.so"),
                       ("STAMP", "lib/stamp.txt")):
        monkeypatch.setattr(_build, name, str(tmp_path / file))
    return src


@pytest.mark.parametrize("why", [RuntimeError("g++ failed: Python.h"), FileNotFoundError("g++")])
def test_the_library_is_built_without_the_host_calls(small_build, monkeypatch, why):
    def fails():
        raise why

    monkeypatch.setattr(_build, "_compile_fast", fails)
    os.makedirs(_build.LIBDIR)
    open(_build.FASTPATH, "w").write("of other sources")
    with pytest.warns(RuntimeWarning, match="_pa_fast.so"):
        path = _build.build()
    assert ctypes.CDLL(path).pa_one() == 1 and not os.path.exists(_build.FASTPATH)
    assert _build.up_to_date()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _build.build()                                        # not tried again with each call
    os.utime(small_build, (2e9, 2e9))
    assert not _build.up_to_date()


def test_a_library_that_has_lost_its_host_calls_is_built_again(small_build, monkeypatch):
    monkeypatch.setattr(_build, "_compile_fast", lambda: "obj")
    monkeypatch.setattr(_build, "_link_fast", lambda obj: open(_build.FASTPATH, "w").close())
    _build.build()
    assert _build.up_to_date()
    os.remove(_build.FASTPATH)
    assert not _build.up_to_date()


def test_a_failing_library_is_an_error(small_build, monkeypatch):
    monkeypatch.setattr(_build, "_compile_fast", lambda: "obj")
    small_build.write_text("not C++")
    with pytest.raises(RuntimeError, match="one.cu"):
        _build.build()


def test_the_stamp_needs_no_torch(monkeypatch):
    def version(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(_build.importlib.metadata, "version", version)
    assert _build._stamp().endswith("torch none")


@pytest.mark.parametrize("content", [None, b"", b"not a library"])
def test_calls_without_the_host_calls_go_through_python(monkeypatch, tmp_path, content):
    path = tmp_path / "_pa_fast.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(_build, "FASTPATH", str(path))
    monkeypatch.setattr(_lib, "_fast", None)
    monkeypatch.setattr(_lib, "load", lambda: types.SimpleNamespace())
    monkeypatch.setattr(ops, "_fast", None)
    made = []
    for name in ("_decode_tree", "_tree_verify", "_keep_kv", "_rope_append_kv"):
        monkeypatch.setattr(ops, name, lambda *a, name=name: made.append((name, len(a))))
    with pytest.warns(RuntimeWarning, match="compiled host calls"):
        ops.pa_decode_tree(*"qkvtcsm", 0.1, 1)
    ops.pa_tree_verify(*"mdtsc", 1)
    ops.pa_keep_kv(*"pscbkv")
    ops.pa_rope_append_kv(*"qkvpskvf")
    assert made == [("_decode_tree", 12), ("_tree_verify", 8), ("_keep_kv", 7), ("_rope_append_kv", 15)]
