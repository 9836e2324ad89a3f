"""The package where the PyTorch binding of the training operators is missing, and
the build of a binding that was made against another torch."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def built():
    import __graft_entry__
    __graft_entry__.build()
    from bit_optimizer_gb300 import build
    return build


def test_the_optimizer_is_there_without_the_binding(built, tmp_path):
    pkg = os.path.join(ROOT, "bit_optimizer_gb300")
    shutil.copytree(pkg, tmp_path / "bit_optimizer_gb300",
                    ignore=shutil.ignore_patterns("csrc", "__pycache__", "*.o", "fp8opt_binding*"))
    code = """
import torch, bit_optimizer_gb300 as bo
from bit_optimizer_gb300 import nn, sharded
assert bo.Fp8AdamW and bo.CastPlan and bo.load()
x = torch.zeros(4, 8)
for call in (lambda: bo.gelu(x), lambda: bo.layer_norm(x, x[0]), lambda: nn.linear(x, x)):
    try:
        call()
    except ImportError as e:
        assert "fp8opt_binding" in str(e)
    else:
        raise SystemExit("no error")
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr


def test_the_binding_is_built_again_for_another_torch(built, monkeypatch):
    calls = []
    monkeypatch.setattr(built, "_compile_binding", lambda: calls.append(1))
    monkeypatch.setattr(built, "_compile", lambda *a: pytest.fail("the library is not stale"))
    built.build()
    assert not calls
    monkeypatch.setattr(built.importlib.metadata, "version", lambda name: "0.1")
    built.build()
    assert calls == [1]
