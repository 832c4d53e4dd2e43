"""The build of _cache_ops.so: left out without torch, anew for another torch."""
import importlib.metadata
import os

import pytest

from prefix_aware_decode_b200 import _build


@pytest.fixture
def here(tmp_path, monkeypatch):
    """A built module of the installed torch, in a folder of its own; what a build would run."""
    calls = []

    def run(cmd):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(_build, "TORCH_OPS", str(tmp_path / "_cache_ops.so"))
    monkeypatch.setattr(_build, "STAMP", str(tmp_path / "made_for"))
    monkeypatch.setattr(_build.subprocess, "check_call", run)
    assert _build.build_torch_ops() == _build.TORCH_OPS
    return calls


def test_the_module_is_built_once(here):
    assert len(here) == 1 and _build.build_torch_ops() == _build.TORCH_OPS and len(here) == 1
    assert _build.build_torch_ops(force=True) and len(here) == 2


def test_the_module_is_built_anew_for_another_torch(here, monkeypatch):
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0")
    assert _build.build_torch_ops() == _build.TORCH_OPS and len(here) == 2
    assert _build.build_torch_ops() and len(here) == 2


def test_without_torch_the_module_is_left_out(here, monkeypatch, capsys):
    def none(name):
        raise importlib.metadata.PackageNotFoundError(name)

    os.unlink(_build.TORCH_OPS)
    monkeypatch.setattr(importlib.metadata, "version", none)
    assert _build.build_torch_ops() is None and len(here) == 1
    assert "not built" in capsys.readouterr().err
