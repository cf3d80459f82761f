"""build(): the library does not hang on the extension module."""
import builtins
import types

import pytest

from hpc_linear_algebra_amd import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """No compiler runs: the library's link is recorded, its sources compile to names."""
    seen = []

    def run(cmd, **_):
        seen.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "_compile", lambda src: src)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libtlrgemm.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    return seen


def test_a_failing_extension_leaves_the_library_built(commands, monkeypatch, tmp_path):
    def fail():
        raise RuntimeError("hipcc failed for binding.cpp")

    monkeypatch.setattr(build, "_build_binding", fail)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert (tmp_path / "libtlrgemm.so").exists()


def test_without_torch_the_library_is_built_alone(commands, monkeypatch, tmp_path, capsys):
    real = builtins.__import__

    def without(name, *args, **kwargs):
        if name.split(".")[0] == "torch":
            raise ImportError("No module named 'torch'", name="torch")
        return real(name, *args, **kwargs)

    monkeypatch.setattr(builtins, "__import__", without)
    assert build.build() == str(tmp_path / "libtlrgemm.so")
    assert (tmp_path / "libtlrgemm.so").exists() and not (tmp_path / "_binding.so").exists()
    assert "torch" in capsys.readouterr().err


def test_both_are_built(commands, tmp_path):
    build.build()
    assert (tmp_path / "libtlrgemm.so").exists() and (tmp_path / "_binding.so").exists()


def test_the_extension_is_host_code(commands):
    """hipcc takes a .cpp for HIP and, unless told, builds device code for an architecture of its own choice."""
    build.build()
    cmd, = [c for c in commands if any(str(a).endswith("binding.cpp") for a in c)]
    assert cmd[cmd.index("-x") + 1] == "c++" and cmd.index("-x") < [str(a).endswith("binding.cpp") for a in cmd].index(True)
