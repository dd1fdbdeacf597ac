"""A block's scale where a row is not finite (tests/kv_scale_check.cu, compiled for the host)."""
import os
import shutil
import subprocess

import pytest

from hybrid_linear_attention_conv_gb300 import build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_marked_scales(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "kv_scale_check")
    r = subprocess.run([nvcc, "-std=c++17", "-O1", *gbuild.ARCH, "-I", gbuild.INCLUDE, "-I", gbuild.CSRC,
                        os.path.join(ROOT, "tests", "kv_scale_check.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "OK" in r.stdout, r.stdout[-2000:]
