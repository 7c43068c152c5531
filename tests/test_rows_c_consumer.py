"""The append and the attentions from plain C (c_consumer/rows.c), with no torch
in the process."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIBDIR = os.path.join(ROOT, "gather_plan_build_amd")
ROCM = "/opt/rocm"


def consumer(tmp_path):
    exe = str(tmp_path / "rows")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror",
                    "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROCM, "include"), "-o", exe,
                    os.path.join(HERE, "c_consumer", "rows.c"),
                    "-L", LIBDIR, "-lgpb", "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-lm",
                    "-Wl,-rpath," + LIBDIR, "-Wl,-rpath," + os.path.join(ROCM, "lib")],
                   check=True)
    return exe


def test_host_side_from_c(tmp_path):
    r = subprocess.run([consumer(tmp_path), "check"], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.gpu
def test_append_and_attend_from_c(tmp_path):
    r = subprocess.run([consumer(tmp_path), "run"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
