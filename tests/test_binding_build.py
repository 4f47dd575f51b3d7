"""The compiled binding beside libloki.so: when it is built anew."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_attention_decode_loki_b200")


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """build.py with its outputs in a folder of the test's and a compiler that writes an empty file; its commands."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "BUILD", str(tmp_path))
    monkeypatch.setattr(mod, "PKG", str(tmp_path))
    monkeypatch.setattr(mod, "BINDING", str(tmp_path / os.path.basename(mod.BINDING)))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(mod.subprocess, "run", run)
    return mod, ran, tmp_path


def test_binding_is_built_once_for_one_torch_and_interpreter(builder):
    mod, ran, _ = builder
    mod.build_binding()
    mod.build_binding()
    assert len(ran) == 1
    mod.build_binding(force=True)
    assert len(ran) == 2


@pytest.mark.parametrize("what", ["torch", "abi", "python", "command", "no stamp"])
def test_binding_is_built_anew(builder, monkeypatch, what):
    mod, ran, folder = builder
    mod.build_binding()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9+cu999")
    elif what == "abi":
        was = torch.compiled_with_cxx11_abi()
        monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: not was)
    elif what == "python":
        monkeypatch.setattr(sys, "version", "3.99.0 (another)")
    elif what == "command":
        monkeypatch.setattr(mod, "ROOT", os.path.join(mod.ROOT, "."))  # (the headers' place)
    else:
        os.remove(folder / "binding.stamp")
    mod.build_binding()
    assert len(ran) == 2
    mod.build_binding()
    assert len(ran) == 2


def test_binding_is_named_after_its_interpreter(builder):
    import sysconfig
    mod, _, folder = builder
    (folder / "_binding.so").write_text("of an earlier build, under a name that any interpreter takes")
    mod.build_binding()
    assert os.path.basename(mod.BINDING) == "_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    assert not (folder / "_binding.so").exists()
