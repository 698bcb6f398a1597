"""What the build and the import need (no GPU, nothing is compiled here)."""
import os
import subprocess
import sys

import pytest

from fp8_block_scaled_02_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    """Commands instead of compilations; outputs, empty, in tmp_path."""
    for name in ("LIB", "ATTN_LIB", "ATTN_BINDING"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    calls, missing = [], set()

    def check_call(cmd):
        if os.path.basename(cmd[0]) in missing:
            raise FileNotFoundError(cmd[0])
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    return tmp_path, calls, missing


def test_everything_is_built(compilers):
    out, calls, _ = compilers
    assert build.build() == build.LIB
    assert sorted(os.listdir(out)) == ["_attn_binding.so", "libfp8attn.so", "libfp8blk.so"]
    assert [os.path.basename(c[0]) for c in calls] == ["hipcc", "hipcc", "g++"]


def test_the_linear_library_needs_hipcc_alone(compilers):
    out, _, missing = compilers
    missing.add("g++")
    with pytest.raises(FileNotFoundError):
        build.build()
    assert (out / "libfp8blk.so").exists()


def test_import_without_a_gpu_build_of_torch():
    """The linear layers' module imports where torch has no device calls; the attention's calls look them up on first
    use."""
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import fp8_block_scaled_02_amd as F\n"
            "F.lib()\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
