"""What the attention kernels' direct loads rest on, in the machine code: they
write m0 without telling the compiler, so no other instruction may use it."""
import importlib.util
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
PACKAGE = os.path.join(os.path.dirname(HERE), "gather_plan_build_amd")


def uses_of_m0(text):
    """(uses within written-out code, the other instructions that name m0)."""
    inside, within, others = False, 0, []
    for line in text.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            inside = "#ASMSTART" in line
        elif re.search(r"\bm0\b", line.split(";")[0]):
            within += inside
            if not inside:
                others.append(line.strip())
    return within, others


def test_only_the_direct_loads_use_m0(tmp_path):
    spec = importlib.util.spec_from_file_location("gpb_build", os.path.join(PACKAGE, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = str(tmp_path / "attend.s")
    flags = [x for x in build.command(out)
             if x not in build.sources() and x not in ("-shared", "-Werror")]
    subprocess.run(flags + ["--offload-device-only", "-S",
                            os.path.join(PACKAGE, "csrc", "attend.hip")],
                   check=True, capture_output=True)
    with open(out) as f:
        within, others = uses_of_m0(f.read())
    assert within > 100 and others == []


def test_a_use_of_m0_is_found():
    text = "\t;;#ASMSTART\n\ts_mov_b32 m0, s4\n\t;;#ASMEND\n\tv_mov_b32 v0, v1 ; m0\n"
    assert uses_of_m0(text) == (1, [])
    assert uses_of_m0(text + "\ts_mov_b32 m0, s1\n") == (1, ["s_mov_b32 m0, s1"])
