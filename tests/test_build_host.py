"""build.py without running a compiler: what it compiles and leaves where the
binding's module can be built, and where it cannot."""
import os
import subprocess
import sys

import pytest

from block_wise_int4_matmulnbits_amd import build as B


@pytest.fixture
def there(tmp_path, monkeypatch):
    """build.py's outputs in tmp_path, its commands recorded and done by writing
    their outputs; a module of older sources lies there."""
    ran = []

    def run(cmd, verbose):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")

    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    for name in ("LIB", "PROBE_LIB", "TORCH_MODULE"):
        monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    (tmp_path / "mnb_torch.so").write_text("old")
    return tmp_path, ran


def _left(path):
    return sorted(p for p in os.listdir(path) if p != "_build")


def test_library_and_module(there):
    path, ran = there
    assert B.build() == B.LIB
    assert _left(path) == ["libmnb.so", "libmnb_probe.so", "mnb_torch.so"]
    assert (path / "mnb_torch.so").read_text() == "new"


def test_library_without_torch(there, monkeypatch, capsys):
    """The C library needs neither torch nor Python's headers."""
    path, ran = there
    monkeypatch.setitem(sys.modules, "torch", None)        # import torch raises ImportError
    assert B.build() == B.LIB
    assert _left(path) == ["libmnb.so", "libmnb_probe.so"]
    assert not any("mnb_torch.cpp" in part for cmd in ran for part in cmd)
    assert "mnb_torch.so" in capsys.readouterr().err


def test_library_where_the_module_does_not_compile(there, monkeypatch, capsys):
    path, ran = there
    run = B._run

    def fails(cmd, verbose):
        run(cmd, verbose)
        if any("mnb_torch.cpp" in part for part in cmd):
            raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(B, "_run", fails)
    assert B.build() == B.LIB
    assert _left(path) == ["libmnb.so", "libmnb_probe.so"]
    assert "mnb_torch.so" in capsys.readouterr().err


def test_library_that_does_not_compile(there, monkeypatch):
    path, ran = there
    run = B._run

    def fails(cmd, verbose):
        if any("mnb_lora.hip" in part for part in cmd):
            raise subprocess.CalledProcessError(1, cmd)
        run(cmd, verbose)

    monkeypatch.setattr(B, "_run", fails)
    with pytest.raises(subprocess.CalledProcessError):
        B.build()
    assert "libmnb.so" not in _left(path)
