"""The native half of the Python cache calls is rebuilt, and not loaded, when the
installed torch is another one than it was built for."""
import os

import pytest
import torch

import block_sparse_local_b200 as sta
from block_sparse_local_b200 import build as sta_build


class _Started:
    """Stands in for a compiler process and records what was started."""
    commands = []
    returncode = 0

    def __init__(self, cmd, **_):
        _Started.commands.append(cmd)

    def communicate(self):
        return "", ""


def test_another_torch_is_noticed(monkeypatch):
    sta_build.build()
    assert sta_build.kv_torch_matches()
    monkeypatch.setattr(sta_build.subprocess, "Popen", _Started)
    monkeypatch.setattr(_Started, "commands", [])
    sta_build.build()
    assert _Started.commands == []                   # everything is up to date
    monkeypatch.setattr(torch, "__version__", "99.0.0")
    sta_build.build()
    (cmd,) = _Started.commands
    assert cmd[0] == "g++" and sta_build.KV_TORCH_SOURCE in cmd
    monkeypatch.setattr(sta, "_KV_TORCH", None)
    with pytest.raises(RuntimeError, match="build it again"):
        sta._kv_torch()


def test_the_loaded_module_is_the_file():
    sta_build.build()
    assert os.path.samefile(sta._kv_torch().__file__, sta_build.KV_TORCH_PATH)
