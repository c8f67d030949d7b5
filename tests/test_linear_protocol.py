"""The waits of the linear attention kernel without a GPU: every order in which its
roles, loads and products may go on, with the kernel's own choice of buffers and
barrier phases (``csrc/linear_protocol.h``), through ``tests/c/linear_protocol_check.cc``."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_order_of_the_roles_sticks_or_reads_what_it_did_not_wait_for(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "linear_protocol_check")
    cmd = [cxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
           "-I", os.path.join(ROOT, "dsa_sparse_attention_03_gb300", "csrc"),
           os.path.join(ROOT, "tests", "c", "linear_protocol_check.cc"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout + run.stderr
    assert run.stdout.strip().endswith("all ok"), run.stdout
