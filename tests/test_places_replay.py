"""Which strided arguments share a byte (CPU): tests/places_replay.cc includes the
rule that the library refuses overlaps by and compares it with sets of bytes on
random small arguments. None that share one may be accepted; none that share none
may be refused where each axis steps over the ones inside."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_overlaps(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / "places_replay")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "ring_allreduce_virtual_gb300", "csrc"),
                    os.path.join(HERE, "places_replay.cc"), "-o", exe], check=True)
    r = subprocess.run([exe, "200000"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("ok")
