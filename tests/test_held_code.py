"""As tests/test_rows_code.py, for the attention of rows held in 8 bits: its direct
loads write m0 without telling the compiler, so no other instruction may use it."""
import importlib.util
import os
import subprocess

from test_rows_code import PACKAGE, uses_of_m0


def test_only_the_direct_loads_use_m0(tmp_path):
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
    assert within > 100 and others == []
