"""The build's parts stand by themselves: the C library where torch or g++ is missing, and the torch form of the 8-bit
operators without its extension."""
import subprocess
import sys
from pathlib import Path

import pytest

from mlp_neural_shading_amd import build as M

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture
def dry(tmp_path, monkeypatch, request):
    """A build whose compilers only write empty files, into a folder of its own with an extension of an earlier build."""
    for name in ("LIB", "CEILING_LIB", "TORCH_LIB"):
        monkeypatch.setattr(M, name, tmp_path / getattr(M, name).name)
    monkeypatch.setattr(M, "BUILD_DIR", tmp_path / "objects")
    M.TORCH_LIB.touch()
    ran = []

    def run(cmd, **_):
        ran.append(cmd)
        fails = getattr(request, "param", None) == "extension fails" and any("mlp_torch_fp8" in c for c in cmd)
        if not fails:
            Path(cmd[cmd.index("-o") + 1]).touch()
        return subprocess.CompletedProcess(cmd, 1 if fails else 0, "", "no such header" if fails else "")
    monkeypatch.setattr(M.subprocess, "run", run)
    return ran


def test_builds_everything(dry):
    M.TORCH_LIB.unlink()
    assert M.build() == M.LIB
    assert M.LIB.exists() and M.CEILING_LIB.exists() and M.TORCH_LIB.exists()


def test_without_torch(dry, monkeypatch, capsys):
    """The library and the probe; the extension of an earlier build, whose structs may be others, goes."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert M.build() == M.LIB
    assert M.LIB.exists() and M.CEILING_LIB.exists() and not M.TORCH_LIB.exists()
    assert not any("g++" in c[0] for c in dry) and "torch" in capsys.readouterr().err


def test_without_a_host_compiler(dry, monkeypatch, capsys):
    monkeypatch.setattr(M.shutil, "which", lambda name: None)
    assert M.build() == M.LIB
    assert M.LIB.exists() and M.CEILING_LIB.exists() and not M.TORCH_LIB.exists()
    assert "g++" in capsys.readouterr().err


@pytest.mark.parametrize("dry", ["extension fails"], indirect=True)
def test_an_extension_that_does_not_compile_is_an_error_of_its_own(dry):
    with pytest.raises(RuntimeError, match="mlp_torch_fp8"):
        M.build()
    assert M.LIB.exists() and M.CEILING_LIB.exists() and not M.TORCH_LIB.exists()


def test_the_torch_form_without_its_extension():
    """Imports, and leaves each call to the checks in Python."""
    code = """if True:
        import sys, torch
        sys.modules["mlp_neural_shading_amd._torch_fp8"] = None
        from mlp_neural_shading_amd import ops_fp8 as E
        f = torch.zeros(4, 130)
        q = E.Quantized(f.to(E.FP8), torch.ones(4, 2))
        for call in (lambda: E.quantize(f), lambda: E.rms_norm(f), lambda: E.linear(q, q)):
            try:
                call()
            except ValueError as e:
                assert "on the GPU" in str(e), e
            else:
                raise SystemExit("not refused")
    """
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
