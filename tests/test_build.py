"""What build() leaves behind where a tool that only the binding's extension module needs is missing. nvcc and the
C++ compiler are stand-ins that write their output file or fail, so that nothing is compiled."""
import os
import warnings

import pytest

from paged_kv_cache_83_gb300 import binding, build as lib_build


def tool(path, works):
    """A compiler: writes what follows -o, or fails with a message."""
    path.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\n: > "$2"\n' if works else '#!/bin/sh\necho no headers >&2\nexit 1\n')
    path.chmod(0o755)
    return str(path)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    monkeypatch.setattr(lib_build, "BUILD", tmp_path / "_build")
    monkeypatch.setattr(lib_build, "LIB", tmp_path / "_build" / "libpagedattn.so")
    monkeypatch.setenv("NVCC", tool(tmp_path / "nvcc", True))
    monkeypatch.setenv("CXX", tool(tmp_path / "g++", True))
    return tmp_path


def test_everything_is_there(tree):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert lib_build.build() == lib_build.LIB
    assert lib_build.LIB.exists() and lib_build.args_path().exists()


@pytest.mark.parametrize("how", ["fails", "missing"])
def test_the_library_needs_no_cpp_compiler(tree, monkeypatch, how):
    monkeypatch.setenv("CXX", tool(tree / "g++2", False) if how == "fails" else str(tree / "none"))
    with pytest.warns(RuntimeWarning, match="no headers" if how == "fails" else "none"):
        assert lib_build.build() == lib_build.LIB
    assert lib_build.LIB.exists() and not lib_build.args_path().exists()


def test_a_module_of_older_sources_does_not_stay(tree, monkeypatch):
    lib_build.build()
    os.utime(lib_build.args_path(), (0, 0))
    monkeypatch.setenv("CXX", tool(tree / "g++2", False))
    with pytest.warns(RuntimeWarning):
        lib_build.build()
    assert not lib_build.args_path().exists()


def test_a_failure_of_nvcc_is_an_error(tree, monkeypatch):
    monkeypatch.setenv("NVCC", tool(tree / "nvcc2", False))
    with pytest.raises(RuntimeError, match="no headers"):
        lib_build.build()


def test_the_calls_say_what_is_missing(tree, monkeypatch):
    monkeypatch.setattr(binding, "_args", None)
    monkeypatch.setattr(binding, "load", lambda: None)
    monkeypatch.setattr(binding, "args_path", lib_build.args_path)
    for call, n in ((binding.pa_rope_store_kv, 9), (binding.pa_chunk_attn, 9), (binding.pa_sample, 2)):
        with pytest.raises(RuntimeError, match="build"):
            call(*[None] * n)
