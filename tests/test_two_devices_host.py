"""The library's launches with more than one device in a process, on the CPU:
its own objects linked against a runtime that only keeps account
(native/two_devices.cpp)."""
import glob
import os
import shutil
import subprocess

import pytest

from long_context_speculative_ds_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_device_allows_the_shared_memory(tmp_path):
    build.build()
    cuda = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    libs = [p for p in (os.path.join(cuda, "lib64"),) if
            os.path.exists(os.path.join(p, "libcudart.so"))]
    if not libs:
        pytest.skip("no shared CUDA runtime to take the kernels' registration")
    exe = str(tmp_path / "two_devices")
    objs = glob.glob(os.path.join(build.OUT_DIR, "_obj", "*.o"))
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + build.INCLUDE,
                        "-I" + os.path.join(cuda, "include"),
                        os.path.join(HERE, "native", "two_devices.cpp"), *objs, "-o", exe,
                        "-L" + libs[0], "-lcudart", "-Wl,-rpath," + libs[0]],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
