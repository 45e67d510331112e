"""What the build makes, in which order and when again (no GPU, no compiler: the commands are recorded)."""
import os
import types

import pytest

from block_quantized_int8_q8_gb300 import _build


@pytest.fixture
def site(monkeypatch, tmp_path):
    """A build in a folder of its own, with commands that write their output file, or fail where `fails` says so."""
    lib = tmp_path / "lib"
    for name, path in (("LIBDIR", lib), ("OBJDIR", tmp_path / "obj"), ("LIB", lib / "libmmq_gb300.so"),
                       ("PEAKS_LIB", lib / "libmmq_peaks.so"), ("BIND_LIB", lib / "_attention.so")):
        monkeypatch.setattr(_build, name, str(path))
    site = types.SimpleNamespace(commands=[], fails=lambda cmd: False, torch="1.2.3+x")

    def run(cmd, **kw):
        site.commands.append(cmd)
        if site.fails(cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "_torch_version", lambda: site.torch, raising=False)
    return site


def binding(cmd):
    return _build.BIND_SRC in cmd or any("_attention.so" in c for c in cmd)


def test_the_library_is_built_without_the_binding_s_headers(site):
    site.fails = binding
    with pytest.raises(RuntimeError, match="attention.cpp"):
        _build.build()
    assert os.path.exists(_build.LIB) and os.path.exists(_build.PEAKS_LIB) and not os.path.exists(_build.BIND_LIB)
    assert not _build.up_to_date()
    site.fails = lambda cmd: False
    del site.commands[:]
    _build.build()
    assert os.path.exists(_build.BIND_LIB) and _build.up_to_date()
    assert all(binding(c) for c in site.commands)              # the library is not made again


def test_the_library_is_built_without_torch(site):
    site.torch = None
    _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BIND_LIB) and _build.up_to_date()
    assert not any(binding(c) for c in site.commands)


def test_another_torch_makes_another_binding(site):
    _build.build()
    assert _build.up_to_date()
    site.torch = "1.2.4+x"
    assert not _build.up_to_date()
    del site.commands[:]
    _build.build()
    assert _build.up_to_date() and site.commands and all(binding(c) for c in site.commands)
