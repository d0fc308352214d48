"""Device code that only the tests need: tests/native/*.cu, each compiled into a library of its own."""
import ctypes
import os
import subprocess

from ternary_weight_dp4a_gb300 import build

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native")


def compile_library(name, directory, *more):
    """Compile native/<name>.cu (and more of the library's sources) and load it."""
    out = os.path.join(str(directory), f"{name}.so")
    cmd = [build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-shared", "-o", out, os.path.join(HERE, f"{name}.cu"),
           *(os.path.join(build.CSRC, m) for m in more)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return ctypes.CDLL(out)
