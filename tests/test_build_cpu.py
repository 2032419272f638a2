"""What the build makes anew: the module that calls the library from Python is bound to PyTorch and Python, the library
to neither."""
import os
import subprocess
import sys

import pytest

from gemm_affine_int4_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """A tree in which everything is up to date; what the build runs is noted, and makes its target."""
    seen = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        seen.append(os.path.basename(out).split(".tmp")[0])
        return Done

    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgai4.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "_torch", lambda: ("/torch", "version one"))
    monkeypatch.setattr(build.subprocess, "run", run)
    build.build()
    assert "torch_calls.o" in seen and seen[-2:] == ["libgai4.so", "_calls.so"]
    seen.clear()
    build.build()
    assert seen == []
    return seen


def test_another_pytorch(commands, monkeypatch):
    monkeypatch.setattr(build, "_torch", lambda: ("/torch", "version two"))
    build.build()
    assert "torch_calls.o" in commands and "_calls.so" in commands and not any(c.startswith("qmm") for c in commands)
    commands.clear()
    build.build()
    assert commands == []


def test_another_python(commands, monkeypatch):
    monkeypatch.setattr(build.sys, "version", sys.version + " of another day")
    build.build()
    assert "torch_calls.o" in commands and "_calls.so" in commands


def test_a_module_that_failed_to_compile_is_compiled_again(commands, monkeypatch):
    monkeypatch.setattr(build, "_torch", lambda: ("/torch", "version two"))
    good = build.subprocess.run

    def run(cmd, **k):
        done = good(cmd, **k)
        if cmd[0] == "g++" and "-c" in cmd:
            return type("Failed", (), dict(returncode=1, stdout="", stderr=""))
        return done

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="torch_calls.cpp"):
        build.build()
    assert "libgai4.so" in commands and "_calls.so" not in commands
    monkeypatch.setattr(build.subprocess, "run", good)
    monkeypatch.setattr(build, "_torch", lambda: ("/torch", "version one"))
    commands.clear()
    build.build()
    assert "torch_calls.o" in commands and "_calls.so" in commands


def test_library_without_pytorch(commands, monkeypatch, capsys):
    monkeypatch.setattr(build, "_torch", lambda: None)
    assert build.build(force=True) == build.LIB
    assert "libgai4.so" in commands and "_calls.so" not in commands and "torch_calls.o" not in commands
    assert "no PyTorch for CUDA" in capsys.readouterr().err


def test_where_pytorch_is_not(monkeypatch, tmp_path):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build._torch() is None
    # one without CUDA
    (tmp_path / "lib").mkdir()
    (tmp_path / "version.py").write_text("cuda = None\n")
    spec = type("Spec", (), dict(origin=str(tmp_path / "__init__.py")))
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)
    assert build._torch() is None
    (tmp_path / "lib" / "libtorch_cuda.so").write_text("")
    assert build._torch() == (str(tmp_path), "cuda = None\n")


def test_why_the_module_does_not_load_is_told():
    program = ("import sys, gemm_affine_int4_gb300 as g4\n"
               "sys.modules['gemm_affine_int4_gb300._calls'] = None\n"
               "try:\n    g4._bind()\nexcept RuntimeError as e:\n    print(e, '|', e.__cause__)\n")
    done = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=120)
    told, cause = done.stdout.strip().split(" | ")
    assert cause and cause in told, done.stdout + done.stderr
