"""The native part of the binding belongs to one PyTorch version: it is
compiled again for another, and not loaded by one."""
import os
import types

import pytest
import torch

from bit_weight_only_g128_gb300 import build as wbuild
from bit_weight_only_g128_gb300 import layer


@pytest.fixture
def compiled(monkeypatch):
    """Commands that would have compiled."""
    wbuild.build_binding()
    ran = []

    def run(cmd, **k):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(wbuild.subprocess, "run", run)
    return ran


def test_compiled_once_for_a_version(compiled):
    assert wbuild.binding_version() == torch.__version__
    wbuild.build_binding()
    assert not compiled


def test_compiled_again_for_another_version(compiled, monkeypatch, tmp_path):
    path = str(tmp_path / "_binding.so")
    for name, p in (("BUILD", str(tmp_path)), ("BINDING", path), ("BINDING_FOR", path + ".torch")):
        monkeypatch.setattr(wbuild, name, p)
    wbuild.build_binding()
    assert len(compiled) == 1 and os.path.exists(path)
    wbuild.build_binding()
    assert len(compiled) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert wbuild.binding_version() != torch.__version__
    wbuild.build_binding()
    assert len(compiled) == 2 and wbuild.binding_version() == "0.0.0"


def test_not_loaded_by_another_version(monkeypatch):
    wbuild.build()
    monkeypatch.setattr(layer, "_native_module", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(ImportError, match="compiled for another PyTorch"):
        layer._native()
