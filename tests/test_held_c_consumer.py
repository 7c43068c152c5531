"""Rows held in e4m3 from plain C (c_consumer/held.c), with no torch in the
process, and what the attention kernels over them rest on in the machine code."""
import importlib.util
import os
import subprocess

import pytest

from test_rows_code import PACKAGE, uses_of_m0

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
ROCM = "/opt/rocm"


def consumer(tmp_path):
    exe = str(tmp_path / "held")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror",
                    "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROCM, "include"), "-o", exe,
                    os.path.join(HERE, "c_consumer", "held.c"),
                    "-L", PACKAGE, "-lgpb", "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-lm",
                    "-Wl,-rpath," + PACKAGE, "-Wl,-rpath," + os.path.join(ROCM, "lib")],
                   check=True)
    return exe


def test_host_side_from_c(tmp_path):
    r = subprocess.run([consumer(tmp_path), "check"], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.gpu
def test_append_read_and_attend_from_c(tmp_path):
    r = subprocess.run([consumer(tmp_path), "run"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr


def test_only_the_direct_loads_use_m0(tmp_path):
    """The direct loads write m0 without telling the compiler: no other instruction
    of the kernels over held rows may use it."""
    spec = importlib.util.spec_from_file_location("gpb_build", os.path.join(PACKAGE, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = str(tmp_path / "attend_held.s")
    flags = [x for x in build.command(out)
             if x not in build.sources() and x not in ("-shared", "-Werror")]
    subprocess.run(flags + ["--offload-device-only", "-S",
                            os.path.join(PACKAGE, "csrc", "attend_held.hip")],
                   check=True, capture_output=True)
    with open(out) as f:
        within, others = uses_of_m0(f.read())
    assert within > 20 and others == []
