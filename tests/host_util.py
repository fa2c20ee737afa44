"""Compiles a small host program against the library's sources and runs it (no GPU)."""

import os
import subprocess

from block_sparse_local_nb_b200.build import CSRC, nvcc


def run_host_program(tmp_path, source: str) -> str:
    src, out = os.path.join(tmp_path, "check.cu"), os.path.join(tmp_path, "check")
    with open(src, "w") as f:
        f.write(source)
    cmd = [nvcc(), "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I" + CSRC, src,
           "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([out], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    return res.stdout
