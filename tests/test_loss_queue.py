"""The queue of the cross entropy's tiles on the host, from the functions that the
kernel itself is compiled from (csrc/loss_queue.cuh)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_tile_once_and_after_what_it_waits_for(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    exe = tmp_path / "queue"
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-I",
                    os.path.join(ROOT, "embedding_lookup_tied_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "loss_queue_model.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe), "1500"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
