"""The layer norm kernels' layouts replayed on the host (CPU):
tests/ln_layout_replay.cu includes the plans and places that the kernels use and
checks coverage, bounds, alignment, shared memory and workspace on random
sizes."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_layouts(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "ln_layout_replay")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O2", "-std=c++17",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "ring_allreduce_virtual_gb300", "csrc"),
                    os.path.join(HERE, "ln_layout_replay.cu"), "-o", exe], check=True)
    r = subprocess.run([exe, "1500"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("ok")
