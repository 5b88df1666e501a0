"""The package without its compiled binding, with one that does not load, and on
a torch without a GPU build (no GPU needed): what went through ctypes still
runs, and the operators of the binding say what is wrong."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "bit_block_scaled_quantize_amd"

USE = """
import torch
{before}
import bit_block_scaled_quantize_amd as nv
assert nv.nvfp4_gemm_workspace_size is not None and nv.nvfp4_quantize_workspace_size(64, 64) > 0
assert nv.nvfp4_route_workspace_size(1, 64) == 0
try:
    nv.nvfp4_rmsnorm(torch.zeros(4, 64), torch.ones(64))
except Exception as e:
    print(type(e).__name__, e)
"""


def use(where, before=""):
    r = subprocess.run([sys.executable, "-c", USE.format(before=before)], cwd=where, capture_output=True, text=True,
                       timeout=300, env=dict(os.environ, PYTHONPATH=str(where)))
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


@pytest.fixture
def package(tmp_path):
    """A copy of the package without the compiled binding."""
    os.makedirs(tmp_path / PACKAGE)
    for f in os.listdir(os.path.join(ROOT, PACKAGE)):
        if f.endswith(".py") or f == "libnvfp4.so":
            shutil.copy(os.path.join(ROOT, PACKAGE, f), tmp_path / PACKAGE / f)
    return tmp_path


def test_without_the_binding(package):
    out = use(package)
    assert out.startswith("ImportError") and "is not built" in out


def test_with_a_binding_that_does_not_load(package):
    (package / PACKAGE / "_native.so").write_bytes(b"no module")
    out = use(package)
    assert out.startswith("ImportError") and "does not load" in out and "_native.so: " in out  # (the loader's own words)


def test_on_a_torch_without_a_gpu_build():
    out = use(ROOT, "del torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream")
    assert out.startswith("ValueError") and "GPU" in out
