"""Builds and runs the test programs of tests/c that include the library's sources."""
from __future__ import annotations

import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(name, tmp_path, device=False):
    """Output of tests/c/<name>.cu; with `device` its kernels are compiled for the GPU, else only as far as
    the host code needs them."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = tmp_path / name
    code = ["-O3", "-gencode", "arch=compute_103a,code=sm_103a"] if device else ["-O1", "-gencode", "arch=compute_103a,code=compute_103a"]
    subprocess.run([nvcc, "-std=c++17", *code, "-o", str(exe), os.path.join(ROOT, "tests", "c", name + ".cu")], check=True,
                   capture_output=True, timeout=600)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    return r.returncode, r.stdout.strip()
