"""build.py's commands (nothing is compiled): the binding follows torch's C++
ABI, and the library is linked also where the binding cannot be built."""
import importlib.util
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module with its outputs in a folder of the test, and the list of
    its commands; a command makes its output, empty."""
    spec = importlib.util.spec_from_file_location(
        "build_under_test", os.path.join(ROOT, "bit_block_scaled_quantize_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    for name, path in (("BUILD", "_build"), ("LIB", "libnvfp4.so"), ("BINDING", "_native.so")):
        monkeypatch.setattr(b, name, str(tmp_path / path))
    monkeypatch.setattr(b, "hipcc", lambda: "hipcc")
    b.commands = commands
    return b


def test_the_binding_follows_torchs_abi(build):
    build.build()
    cmd = [c for c in build.commands if any(a.endswith("binding.cpp") for a in c)]
    assert len(cmd) == 1 and f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}" in cmd[0]
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)


def test_the_library_is_built_without_a_binding(build, monkeypatch):
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
