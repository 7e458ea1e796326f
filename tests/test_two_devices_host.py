"""The library's launches, on the CPU: its own objects linked against a
runtime of two devices that only keeps account (native/two_devices.cpp)."""
import os
import shutil
import subprocess

import pytest

from long_context_speculative_ds_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    objs = [os.path.join(build.OUT_DIR, "_obj", s + ".o") for s in build.SOURCES]
    build.build(force=not all(os.path.exists(o) for o in objs))
    cuda = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    libs = os.path.join(cuda, "lib64")
    if not os.path.exists(os.path.join(libs, "libcudart.so")):
        pytest.skip("no shared CUDA runtime to take the kernels' registration")
    out = str(tmp_path_factory.mktemp("native") / "two_devices")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + build.INCLUDE,
                        "-I" + os.path.join(cuda, "include"),
                        os.path.join(HERE, "native", "two_devices.cpp"), *objs, "-o", out,
                        "-L" + libs, "-lcudart", "-Wl,-rpath," + libs],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


def _run(*cmd):
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


def test_every_device_allows_the_shared_memory(exe):
    _run(exe)


def test_grids_of_large_batches(exe):
    _run(exe, "batches")
