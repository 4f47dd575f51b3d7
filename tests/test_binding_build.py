"""The compiled binding beside libloki.so: when it is built anew, and what the package does where it cannot be used."""
from __future__ import annotations

import importlib.util
import os
import shutil
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


USE = """
import torch, sparse_attention_decode_loki_b200 as loki
assert loki.dense_decode_workspace_size(1, 8, 8, 4096, 128) > 0  # (libloki.so alone)
assert loki.dense_decode_paged_q8_workspace_size(1, 8, 8, 16, 9, 128) > 0
q = torch.zeros(1, 1, 128)
try:
    loki.loki_decode_attention(q, q[None], q[None], q, 1, 32, 1)
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("CPU tensors were taken")
b = q.view(1, 1, 1, 128)
for call in (lambda: loki.loki_append_keys_paged_rope(b, b, None, b, b, q, q),
             lambda: loki.loki_append_keys_paged_q8(b, b, None, b, b, q, q, q, q),
             lambda: loki.dense_decode_attention_paged_q8(q, b, b, q, q, q, q),
             lambda: loki.loki_sparse_attention_paged_q8(q, b, b, q, q, q, q, q),
             lambda: loki.loki_decode_attention_paged_q8(q, b, b, q, q, b, q, q, q, 16, 1)):
    try:
        call()
    except ImportError as e:
        assert WHY in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError("a call went through without the binding")
"""


def run_copy(tmp_path, code, with_binding):
    """`code` in a new process that sees a copy of the package, with or without its binding."""
    to = tmp_path / "sparse_attention_decode_loki_b200"
    to.mkdir()
    for f in os.listdir(PKG):
        if f.endswith(".py") or (with_binding and f.startswith("_binding")):
            shutil.copy(os.path.join(PKG, f), to / f)
    os.symlink(os.path.join(PKG, "libloki.so"), to / "libloki.so")
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_package_without_its_binding(tmp_path):
    run_copy(tmp_path, "WHY = '_binding'\n" + USE, with_binding=False)


def test_binding_of_another_torch_is_not_used(tmp_path):
    run_copy(tmp_path, "import torch\ntorch.__version__ = '9.9.9+cu999'\nWHY = 'built for torch'\n" + USE, with_binding=True)


def test_binding_that_does_not_load(tmp_path):
    run_copy(tmp_path, "WHY = 'undefined symbol'\nimport importlib.machinery as m\n"
             "def broken(self, spec):\n"
             "    if spec.name.endswith('_binding'):\n"
             "        raise ImportError('undefined symbol: of another torch')\n"
             "    return create(self, spec)\n"
             "create, m.ExtensionFileLoader.create_module = m.ExtensionFileLoader.create_module, broken\n" + USE, with_binding=True)


def test_package_under_a_torch_without_cuda(tmp_path):
    run_copy(tmp_path, "import torch\ndel torch._C._cuda_getCurrentRawStream\n"
             "import sparse_attention_decode_loki_b200 as loki\n"
             "q = torch.zeros(1, 1, 128)\n"
             "try:\n    loki.loki_decode_attention(q, q[None], q[None], q, 1, 32, 1)\n"
             "except ValueError:\n    pass\n", with_binding=True)
