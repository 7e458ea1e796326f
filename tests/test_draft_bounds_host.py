"""What the draft cache's launches and kernels may rely on, checked without a
GPU: places read back from a workspace, and the shared memory that a kernel may
use when calls of several threads meet, and the clusters that a device can place."""
import os
import shutil
import subprocess

import pytest
import torch

from long_context_speculative_ds_gb300 import binding as B
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


def _run_library(tmp_path, source):
    """The library's own objects over a runtime that only keeps account."""
    objs = [os.path.join(build.OUT_DIR, "_obj", s + ".o") for s in build.SOURCES]
    build.build(force=not all(os.path.exists(o) for o in objs))
    libs = os.path.join(CUDA, "lib64")
    if not os.path.exists(os.path.join(libs, "libcudart.so")):
        pytest.skip("no shared CUDA runtime to take the kernels' registration")
    _run(tmp_path, source, *objs, "-L" + libs, "-lcudart", "-Wl,-rpath," + libs)


def test_no_call_takes_shared_memory_from_another(tmp_path):
    _run_library(tmp_path, "draft_allowance.cpp")


def test_clusters_that_a_device_can_place(tmp_path):
    _run_library(tmp_path, "draft_clusters.cpp")


def test_pieces_that_a_workspace_can_name(tmp_path):
    _run(tmp_path, "draft_pieces.cpp")


def test_one_row_of_any_stride():
    """A row by itself has no next one: its buffer's stride does not matter."""
    wide = torch.zeros(3, 8 * 64 + 4, dtype=torch.bfloat16)
    pos, ws = torch.zeros(1, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    row = wide[:1].as_strided((1, 4, 64), (516, 64, 1))
    a = B.rope_append_args(row, None, None, pos, q_out=row, rope_base=1e4, workspace=ws)
    assert (a.q_row_stride, a.q_out_row_stride) == (256, 256)
    two = wide[:2, :4 * 64].unflatten(1, (4, 64))
    pos = torch.zeros(2, dtype=torch.int32)
    a = B.rope_append_args(two, None, None, pos, q_out=two, rope_base=1e4, workspace=ws)
    assert (a.q_row_stride, a.q_out_row_stride) == (516, 516)
