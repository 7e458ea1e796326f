"""What the draft cache's launches and kernels may rely on, checked without a
GPU: places read back from a workspace."""
import os
import shutil
import subprocess

import pytest

from long_context_speculative_ds_gb300 import build

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native")
CUDA = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))


def _run(tmp_path, source, *more):
    out = str(tmp_path / os.path.splitext(source)[0])
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + build.INCLUDE, "-I" + build.CSRC,
                        "-I" + os.path.join(CUDA, "include"), os.path.join(HERE, source), *more,
                        "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([out], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


def test_pieces_that_a_workspace_can_name(tmp_path):
    _run(tmp_path, "draft_pieces.cpp")
