"""What building and loading needs: the C ABI nothing but nvcc, the tensor
operators' module the torch that it is compiled against."""
import os
import subprocess
import sys

import pytest
import torch

from bit_diffusion_transformer_w4a4_b200 import build, svdq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_without_torch_and_cxx():
    """build() and lib() neither import torch nor compile against it."""
    code = """
import sys
sys.modules["torch"] = None            # import torch raises ImportError
from bit_diffusion_transformer_w4a4_b200 import build, svdq
build.bind_stale = lambda: True
build.build()
print(svdq.lib().svdq_version().decode())
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, "CXX": "/nonexistent/c++"},
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    assert "sm_100a" in r.stdout


@pytest.mark.parametrize("version", ["2.11.1", "0.0.0+other"])
def test_module_of_another_torch_is_not_loaded(monkeypatch, version):
    svdq._bind()
    assert not build.bind_stale()
    monkeypatch.setattr(torch, "__version__", version)
    assert build.bind_stale()
