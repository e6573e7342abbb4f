"""The library's build: libember.so alone needs neither torch nor the extension's compiler, and the
torch extension is made again for another torch.  Compilers are stood in for; nothing is compiled."""
import subprocess
import types

import pytest
import torch

from gqa_transformer_decode_gb300 import build as B


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """Commands that a build in an empty folder runs; each makes its output file."""
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(B, "OUT", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libember.so"))
    monkeypatch.setattr(B, "TORCH_EXT", str(tmp_path / "paged_torch.so"))
    return ran


def of_ext(ran):
    return [c for c in ran if B.TORCH_SRC in c]


def test_the_library_builds_without_torch(commands, monkeypatch):
    def no_torch(*_):
        raise RuntimeError("no torch headers, no g++")
    monkeypatch.setattr(B, "build_ext", no_torch)
    assert B.build() == B.LIB and commands and not of_ext(commands)
    n = len(commands)
    assert B.up_to_date() and B.build() == B.LIB and len(commands) == n
    B.build(force=True)
    assert len(commands) == 2 * n and not of_ext(commands)


def test_the_extension_is_made_again_for_another_torch(commands, monkeypatch):
    for _ in range(2):
        assert B.build_ext() == B.TORCH_EXT and len(commands) == 1
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert not B.ext_up_to_date()
    for _ in range(2):
        B.build_ext()
        assert B.ext_up_to_date() and len(commands) == 2
    monkeypatch.setattr(torch, "__file__", "/elsewhere/torch/__init__.py")
    B.build_ext()
    assert len(commands) == 3


def test_build_all_makes_both(commands):
    B.build_all()
    assert len(of_ext(commands)) == 1 and any(B.LIB in " ".join(c) for c in commands)
    assert B.up_to_date() and B.ext_up_to_date()
