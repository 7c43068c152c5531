"""Work lists checked by the functions that the attention kernels use
(attend.h), compiled for the host."""
import ctypes
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def library(path):
    so = str(path / "list_check.so")
    subprocess.run(["/opt/rocm/llvm/bin/clang++", "-std=c++17", "-O1", "-fPIC", "-shared",
                    "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(ROOT, "include"), "-isystem", "/opt/rocm/include",
                    "-I", os.path.join(ROOT, "gather_plan_build_amd", "csrc"),
                    "-o", so, os.path.join(HERE, "list_check.cpp")], check=True)
    return ctypes.CDLL(so)


def outcome(call, plan, lst):
    """(what `call` of the library says of a list, and the item it says it of)."""
    at = ctypes.c_int32(-1)
    return call(ctypes.byref(plan), ctypes.c_void_p(lst.ctypes.data), ctypes.byref(at)), at.value
