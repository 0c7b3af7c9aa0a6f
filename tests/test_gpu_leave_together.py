"""The shared decision to give up in the kernel for few rows: threads that meet at a barrier of fixed size leave in
the same round, whenever a thread outside it raises the flag.  (A kernel in which they did not would wait for ever, so
what is run is the barrier alone, in loops that end by themselves.)"""
import ctypes
import os
import subprocess

import pytest
import torch

from conftest import REPO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def walk(cuda_lib, tmp_path_factory):
    import __graft_entry__
    bm = __graft_entry__.build_module()
    out = str(tmp_path_factory.mktemp("vote") / "libvote.so")
    r = subprocess.run([bm._nvcc()] + bm.NVCC_FLAGS + ["-shared", "-I", bm.INCLUDE, "-I", bm.CSRC,
                       os.path.join(REPO, "tests", "barrier_any_harness.cu"), "-o", out, "-cudart", "shared",
                       "-Xlinker", "-rpath,/usr/local/cuda/lib64"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    lib = ctypes.CDLL(out)
    lib.run_walk.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p]
    return lib.run_walk


@pytest.mark.parametrize("delay", [0, 100, 1234, 20000])
def test_all_leave_in_one_round(walk, delay):
    blocks, rounds = 608, 20000
    left = torch.full((blocks, 512), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert walk(blocks, rounds, delay, left.data_ptr()) == 0
    first = left[:, :1]
    assert bool((left == first).all()) and bool((first >= 0).all()) and bool((first < rounds).all())
