"""What build() does about the compiled binding beside the library, with stand-ins for
the compilers (nothing is compiled)."""
import os

import pytest

from online_softmax_attn_gb300 import build as b


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """build() in an empty folder; returns the names of what it compiled or linked."""
    done = []

    def touch(path, what):
        with open(path, "w") as f:
            f.write(what)
        done.append(what)

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        touch(cmd[cmd.index("-o") + 1], "library")
        return Done

    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "build"))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "CALLS_PATH", str(tmp_path / "calls.so"))
    monkeypatch.setattr(b, "nvcc_path", lambda: "nvcc")
    monkeypatch.setattr(b, "_compile", lambda src, obj, *a: touch(obj, os.path.basename(src)) or "")
    monkeypatch.setattr(b, "_compile_calls", lambda src, out: touch(out, "binding") or "")
    monkeypatch.setattr(b.subprocess, "run", run)
    return done


def test_the_library_is_linked_without_the_binding(sandbox, monkeypatch):
    def fail(src, out):
        raise RuntimeError("no Python.h")

    works = b._compile_calls
    monkeypatch.setattr(b, "_compile_calls", fail)
    with pytest.raises(RuntimeError, match="no Python.h"):
        b.build()
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.CALLS_PATH)
    with pytest.raises(RuntimeError, match="no Python.h"):  # and again: nothing is taken for built
        b.build()
    monkeypatch.setattr(b, "_compile_calls", works)
    del sandbox[:]
    b.build()
    assert sandbox == ["binding"]


def test_the_binding_is_compiled_again_for_another_torch(sandbox, monkeypatch):
    import torch

    b.build()
    assert sorted(sandbox) == sorted([*b.SOURCES, "library", "binding"])
    del sandbox[:]
    b.build()
    assert sandbox == []
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    b.build()
    assert sandbox == ["binding"]
    b.build()
    assert sandbox == ["binding"]


def test_shared_stall_selftest_is_debug_only():
    """The release library refuses it without touching the device."""
    import online_softmax_attn_gb300 as attn

    b.build()
    lib = attn.library()
    assert lib.attn_selftest_shared_stall(2, 0) == lib.attn_selftest_shared_stall(-1, 2) == attn.ATTN_ERR_UNSUPPORTED
    assert lib.attn_selftest_shared_stall(0, 3) == lib.attn_selftest_shared_stall(0, -1) == attn.ATTN_ERR_INVALID_ARG
