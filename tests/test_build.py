"""CPU tests of the build: the library is built wherever nvcc is, with or without the Python
side's extension module.  The compilers are stand-ins that log their calls."""
import importlib.util
import os
import subprocess
import sysconfig

import pytest

import chunked_prefill_mixed_gb300 as S
from chunked_prefill_mixed_gb300 import build as B


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Sets the stand-ins up; returns what runs the build and gives (library there,
    module there, compilers called)."""
    log = tmp_path / "log"
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libsarathi.so"))
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "_paged_calls.so"))

    def tool(name, status):
        path = tmp_path / name
        path.write_text(f"#!/bin/sh\necho {name} >> {log}\n" + "[ %d = 0 ] || exit 1\n" % status +
                        'while [ $# -gt 1 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n')
        path.chmod(0o755)
        return str(path)

    def run(nvcc=0, gxx=0, headers=True, **kw):
        where = tool("nvcc", nvcc)
        monkeypatch.setattr(B, "nvcc", lambda: where)
        tool("g++", gxx)
        monkeypatch.setenv("PATH", str(tmp_path) + os.pathsep + os.environ["PATH"])
        if not headers:
            monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
        log.write_text("")
        error = None
        try:
            B.build(**kw)
        except subprocess.CalledProcessError as e:
            error = e
        return os.path.exists(B.LIB), os.path.exists(B.CALLS), sorted(log.read_text().split()), error
    return run


needs_torch = pytest.mark.skipif(importlib.util.find_spec("torch") is None, reason="no torch")


@needs_torch
def test_both_are_built_once(tools):
    assert tools() == (True, True, ["g++", "nvcc"], None)
    assert tools() == (True, True, [], None)
    assert tools(force=True) == (True, True, ["g++", "nvcc"], None)


@needs_torch
def test_the_library_is_built_where_the_module_cannot_be(tools, tmp_path):
    assert tools(headers=False) == (True, False, ["nvcc"], None)
    assert B.calls_need() == "Python's headers"


@needs_torch
def test_the_library_is_in_place_where_the_module_fails(tools):
    lib, module, called, error = tools(gxx=1)
    assert lib and not module and called == ["g++", "nvcc"] and os.path.basename(error.cmd[0]) == "g++"
    assert tools(gxx=1, calls=False) == (True, False, [], None)


def test_a_library_that_fails_is_an_error(tools):
    lib, module, called, error = tools(nvcc=1)
    assert not lib and "nvcc" in error.cmd[0]


@needs_torch
def test_loading_the_library_does_not_need_the_module(tools, monkeypatch):
    """The step's calls load the library alone; the paged ones say what is missing."""
    tools(headers=False)
    os.remove(B.LIB)
    monkeypatch.setattr(S, "_lib", None)
    monkeypatch.setattr(S, "_calls", None)
    monkeypatch.setattr(B, "stale", lambda *a: True)
    monkeypatch.setattr(S.ctypes, "CDLL", lambda path: (_ for _ in ()).throw(OSError("loaded " + path)))
    with pytest.raises(OSError, match="libsarathi.so"):
        S.load()
    with pytest.raises(ImportError, match="Python's headers"):
        S.paged_calls()


@needs_torch
def test_the_module_is_built_again_for_another_torch_or_python(monkeypatch):
    import importlib.metadata
    import torch
    now = B.calls_path()
    assert now == B.CALLS and os.path.dirname(now) == os.path.dirname(B.LIB)
    assert torch.__version__.split("+")[0] in now
    real = importlib.metadata.version
    with monkeypatch.context() as m:
        m.setattr(importlib.metadata, "version", lambda name: "99.1" if name == "torch" else real(name))
        assert B.calls_path() != now
    with monkeypatch.context() as m:
        m.setattr(B.sys.implementation, "cache_tag", "cpython-399")
        assert B.calls_path() != now
