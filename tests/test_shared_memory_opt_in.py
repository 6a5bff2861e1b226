"""First calls of one kernel from two host threads at once, with different amounts of shared memory:
each gets what it asked for, then and later.  No GPU: the library's object file is linked to a
runtime of tests/shared_memory_opt_in.cpp's own, which decides who comes first."""
import os
import subprocess

import pytest

from block_scaled_mxfp4_gb300 import build as mxbuild


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    mxbuild.build()
    obj = os.path.join(mxbuild.OBJDIR, "layer_norm.cu.o")
    if not os.path.exists(obj):
        mxbuild.build(force=True)                          # (a library that came without its objects)
    exe = str(tmp_path_factory.mktemp("opt_in") / "opt_in")
    src = __file__.replace("test_shared_memory_opt_in.py", "shared_memory_opt_in.cpp")
    cuda = os.path.join(os.path.dirname(os.path.dirname(mxbuild.nvcc())), "include")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-I" + cuda, src, obj, "-o", exe, "-pthread"])
    return exe


@pytest.mark.parametrize("order", ["first", "last"])
def test_two_threads_first_calls(program, order):
    r = subprocess.run([program, order], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
