"""The Python binding's build (no GPU): a module built for one PyTorch is not taken for another's, and the C
library builds without any."""
import os
import sys

import pytest


@pytest.fixture()
def compiled(monkeypatch):
    """build.build_binding with the compiler replaced by one that writes an empty file; the files it made."""
    from video_dit_full_b200 import build
    made = []

    def compiler(cmd):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        made.append(cmd)
    monkeypatch.setattr(build.subprocess, "check_call", compiler)
    return made


def test_another_torch_gets_another_module(built, compiled, monkeypatch):
    import torch
    from video_dit_full_b200 import build, wan_attn
    here = wan_attn.binding_path()
    assert os.path.exists(here) and build.build_binding() == here and not compiled      # up to date
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    other = wan_attn.binding_path()
    assert other != here and not os.path.exists(other)
    monkeypatch.setattr(wan_attn, "_bound", None)
    with pytest.raises(RuntimeError, match="is missing"):                               # not the one that is there
        wan_attn._binding()
    try:
        assert build.build_binding() == other and len(compiled) == 1 and os.path.exists(other)
    finally:
        os.remove(other)
    assert os.path.getsize(here) > 0


def test_binding_loads(built):
    from video_dit_full_b200 import wan_attn
    assert wan_attn._binding().__file__ == wan_attn.binding_path()


def test_library_builds_without_torch(built, compiled, monkeypatch, capsys):
    from video_dit_full_b200 import build
    monkeypatch.setitem(sys.modules, "torch", None)                # import torch raises ImportError
    assert build.build_binding(force=True) is None and not compiled
    assert build.build() == built and "no PyTorch" in capsys.readouterr().err
