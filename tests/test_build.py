"""The build of the torch module of the operators (no GPU, nothing is compiled here)."""
import os
import sys
from types import SimpleNamespace

import pytest

from vla_flow_matching_denoise_b200 import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The commands that would compile; OPS is a file of the test."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        key = [c for c in cmd if c.startswith("-DFM_OPS_BUILT_FOR=")][0].split('"')[1]
        with open(out, "wb") as f:
            f.write(b"\x7fELF" + key.encode() + b"\0")
        return SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "OPS", str(tmp_path / "_ops.so"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def _torch(monkeypatch, version, cuda="12.8"):
    torch = pytest.importorskip("torch")
    fake = SimpleNamespace(__file__=torch.__file__, __version__=version, version=SimpleNamespace(cuda=cuda), _C=torch._C)
    monkeypatch.setitem(sys.modules, "torch", fake)


@pytest.mark.parametrize("kind", ["none", "cpu"])
def test_without_a_cuda_torch_the_library_is_still_built(monkeypatch, compiled, capsys, kind):
    if kind == "none":
        monkeypatch.setitem(sys.modules, "torch", None)           # import torch raises
    else:
        _torch(monkeypatch, "2.11.0+cpu", None)
    monkeypatch.setattr(build, "_build_lib", lambda force, verbose: build.LIB)
    assert build.build(force=True) == build.LIB
    assert not compiled and not os.path.exists(build.OPS)
    assert "_ops.so" in capsys.readouterr().err


def test_the_module_is_built_again_for_another_torch_or_python(monkeypatch, compiled):
    _torch(monkeypatch, "2.11.0")
    build._build_ops(False)
    build._build_ops(False)
    assert len(compiled) == 1
    _torch(monkeypatch, "2.11.01")              # (the first is a prefix of it)
    build._build_ops(False)
    assert len(compiled) == 2
    _torch(monkeypatch, "2.11.0")
    build._build_ops(False)
    assert len(compiled) == 3
    monkeypatch.setattr(sys, "implementation", SimpleNamespace(**{**vars(sys.implementation), "cache_tag": "cpython-399"}))
    build._build_ops(False)
    assert len(compiled) == 4
    os.utime(build.OPS, (1, 1))                 # older than its sources
    build._build_ops(False)
    assert len(compiled) == 5


def test_the_built_module_says_what_it_was_built_for():
    torch = pytest.importorskip("torch")
    if torch.version.cuda is None:
        pytest.skip("needs a CUDA build of torch")
    from vla_flow_matching_denoise_b200 import ops
    assert ops._ops.built_for == f"fm_ops for {sys.implementation.cache_tag}, torch {torch.__version__}"
