"""What build() makes, with the compilers replaced by one that writes its output."""
import builtins
import os
import subprocess
import sys

import pytest

from block_sparse_attention_queries_b200 import build as abbuild


class _Compiler:
    def __init__(self, missing=(), failing=()):
        self.missing, self.failing, self.ran = missing, failing, []

    def __call__(self, cmd, *args, **kw):
        name = os.path.basename(cmd[0])
        if name in self.missing:
            raise FileNotFoundError(cmd[0])
        self.ran.append(name)
        self.returncode = int(name in self.failing)
        if not self.returncode:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write(" ".join(cmd))
        done = type("Process", (), {})()
        done.returncode = self.returncode
        done.wait = lambda: done.returncode
        return done


@pytest.fixture
def made(tmp_path, monkeypatch):
    """Runs build() with both libraries in an empty folder; their names that are there afterwards."""
    monkeypatch.setattr(abbuild, "LIB", str(tmp_path / "libab.so"))
    monkeypatch.setattr(abbuild, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(abbuild, "nvcc", lambda: "nvcc")

    def run(compiler, **kw):
        monkeypatch.setattr(subprocess, "Popen", compiler)
        error = None
        try:
            abbuild.build(**kw)
        except Exception as e:  # noqa: BLE001
            error = e
        return sorted(os.listdir(tmp_path)), error
    return run


def _hide_torch(monkeypatch):
    real = builtins.__import__

    def fake(name, *args, **kw):
        if name.split(".")[0] == "torch":
            raise ImportError(name)
        return real(name, *args, **kw)
    monkeypatch.setattr(builtins, "__import__", fake)
    monkeypatch.delitem(sys.modules, "torch", raising=False)


def test_without_torch_the_library_is_built(made, monkeypatch):
    _hide_torch(monkeypatch)
    compiler = _Compiler()
    assert made(compiler) == (["libab.so"], None) and compiler.ran == ["nvcc"]
    assert made(compiler) == (["libab.so"], None) and compiler.ran == ["nvcc"]   # and nothing more to do
    assert made(compiler, force=True)[1] is None and compiler.ran == ["nvcc"] * 2


@pytest.mark.parametrize("missing,failing,left", [(("g++",), (), ["libab.so"]), ((), ("g++",), ["libab.so"]), (("nvcc",), (), ["_marshal.so"]),
                                                  ((), ("nvcc",), ["_marshal.so"])])
def test_one_failure_leaves_the_other_library(made, missing, failing, left):
    pytest.importorskip("torch")
    names, error = made(_Compiler(missing, failing))
    assert names == left and isinstance(error, FileNotFoundError if missing else subprocess.CalledProcessError)


def test_another_torch(made, monkeypatch):
    torch = pytest.importorskip("torch")
    compiler = _Compiler()
    assert made(compiler)[0] == ["_marshal.so", "libab.so"] and compiler.ran == ["nvcc", "g++"]
    with open(abbuild.MARSHAL, "w") as f:
        f.write(f"AB_TORCH={torch.__version__};")
    assert made(compiler)[1] is None and compiler.ran == ["nvcc", "g++"]
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert made(compiler)[1] is None and compiler.ran == ["nvcc", "g++", "g++"]


def test_the_binding_refuses_checks_for_another_torch(monkeypatch):
    torch = pytest.importorskip("torch")
    import block_sparse_attention_queries_b200 as ab
    abbuild.build()
    assert ab._m().built_for == f"AB_TORCH={torch.__version__};"
    monkeypatch.setattr(ab, "_marshal_module", None)
    monkeypatch.setattr(torch, "__version__", "99.0")
    with pytest.raises(RuntimeError, match="another torch"):
        ab._m()
