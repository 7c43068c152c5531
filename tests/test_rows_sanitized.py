"""The append's and the attentions' host code under AddressSanitizer and
UndefinedBehaviorSanitizer: their argument checks and the work lists of
test_rows_host.py, in a child pytest on a library whose host pass alone is
instrumented.  No call reaches a kernel launch."""
import glob
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "gather_plan_build_amd", "csrc")


def test_rows_host_checks_pass_under_asan_and_ubsan(tmp_path):
    runtimes = sorted(glob.glob(
        "/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not runtimes:
        pytest.skip("no clang AddressSanitizer runtime under /opt/rocm/llvm")
    so = str(tmp_path / "libgpb_san.so")
    cmd = ["hipcc", "--offload-arch=gfx950", "-mcode-object-version=5", "-O1", "-g",
           "-std=c++17", "-fPIC", "-shared",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all",
           "-Xarch_host", "-fno-omit-frame-pointer", "-shared-libsan",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", so]
    subprocess.run(cmd + sorted(glob.glob(os.path.join(CSRC, "*.hip"))), check=True,
                   capture_output=True)
    env = dict(os.environ, GPB_LIB=so, LD_PRELOAD=runtimes[-1],
               ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(HERE, "test_rows_host.py")],
                       env=env, capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
