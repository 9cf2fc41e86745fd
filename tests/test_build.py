"""What the build leaves behind, with compilers that only write the files they are
asked for."""
import os
import stat

import pytest

from exact_attention_67_gb300 import build as b


def script(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


WRITES = 'while [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo made > "$2"; fi; shift; done\n'


@pytest.fixture
def out(tmp_path, monkeypatch):
    monkeypatch.setattr(b, "OUT_DIR", str(tmp_path / "out"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "out" / "libexattn.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "out" / "_exattn_binding.so"))
    monkeypatch.setenv("NVCC", script(tmp_path / "nvcc", WRITES))
    monkeypatch.setenv("CXX", script(tmp_path / "g++", WRITES))
    return tmp_path


def test_the_library_is_built_where_the_binding_cannot_be(out, monkeypatch):
    script(out / "g++", "echo no such compiler >&2; exit 1\n")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING) and not b.up_to_date()

    def no_headers():
        raise ImportError("torch")

    os.remove(b.LIB)
    monkeypatch.setattr(b, "_binding_flags", no_headers)
    with pytest.raises(ImportError):
        b.build()
    assert os.path.exists(b.LIB)


def test_built_once(out):
    assert not b.up_to_date()
    assert b.build() == b.LIB and os.path.exists(b.BINDING) and b.up_to_date()


def test_another_python_or_pytorch_builds_again(out, monkeypatch):
    import torch

    from exact_attention_67_gb300 import paged
    b.build()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not b.up_to_date()
    monkeypatch.setattr(paged, "_binding", None)
    monkeypatch.setattr(paged, "load", lambda: None)
    with pytest.raises(ImportError, match="another"):
        paged._native()
    b.build()
    assert b.up_to_date()
    os.remove(b.BINDING + ".for")
    assert not b.up_to_date()
