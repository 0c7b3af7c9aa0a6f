"""The end of C's rows in the dense products: a TMA store clips at 16 bytes, so rows of any other length are stored
element by element, and the padding of a row keeps what it held (the header: "columns N..ldc-1 are never written")."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import oracle
import workloads as wl
from conftest import REPO


@pytest.fixture(scope="module")
def c_map_ok(tmp_path_factory):
    import __graft_entry__
    __graft_entry__.build()
    bm = __graft_entry__.build_module()
    lib_dir = os.path.dirname(bm.LIB_PATH)
    out = str(tmp_path_factory.mktemp("c_map") / "libc_map.so")
    r = subprocess.run([bm._nvcc()] + bm.ARCH_FLAGS + [
        "-O1", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", bm.INCLUDE, "-I", bm.CSRC,
        os.path.join(REPO, "tests", "c_map_harness.cu"), "-o", out, "-L", lib_dir, "-lgemm_gb300", "-cudart", "shared",
        "-Xlinker", f"-rpath,{lib_dir}:/usr/local/cuda/lib64"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    lib = ctypes.CDLL(out)
    lib.c_map_ok.argtypes = [ctypes.c_ulonglong, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    return lib.c_map_ok


@pytest.mark.parametrize("es", [2, 4])
def test_boxes_only_for_rows_of_whole_16_bytes(c_map_ok, es):
    per = 16 // es
    for N in range(1, 4 * per + 1):
        ldc = -(-N // per) * per + per
        assert c_map_ok(1 << 20, N, ldc, es) == (N % per == 0)
        assert not c_map_ok((1 << 20) + 8, N, ldc, es) and not c_map_ok(1 << 20, N, ldc + 1, es)


@pytest.mark.gpu
@pytest.mark.parametrize("order", [1, 2], ids=["given", "transposed"])
@pytest.mark.parametrize("layout", ["NN", "NT"])
@pytest.mark.parametrize("N", [249, 250, 252, 500, 1023, 1016])
@pytest.mark.parametrize("ab,out", [(wl.F16, wl.F16), (wl.BF16, wl.BF16), (wl.BF16, wl.F32), (wl.F32, wl.F32)],
                         ids=["f16", "bf16", "bf16-f32", "tf32x3"])
def test_padding_stays_at_an_aligned_pitch(cuda_lib, ab, out, N, layout, order):
    """run_gemm holds the padding and the guards around C to their canaries; the integer sums are exact."""
    import torch
    from gpu_util import run_gemm
    g = cuda_lib
    per = 16 // (4 if out == wl.F32 else 2)
    p = wl.random_problem(N, 300, N, 128, ab, out, layout=layout, alpha=2.0, beta=-1.0, integer=True,
                          lda_pad=0, ldb_pad=-N % 8 if layout == "NN" else 0, ldc_pad=-N % per + per)
    assert p.ldc % per == 0
    g.gemm_set_tile_policy(g.TILE_PAIR, 256)
    g.gemm_set_operand_order(order)
    try:
        r = run_gemm(g, p)
    finally:
        g.gemm_set_operand_order(g.ORDER_AUTO)
        g.gemm_set_tile_policy(g.TILE_AUTO, 0)
    info = g.gemm_last_launch()
    assert r.status == 0 and info["path"] == g.PATH_TCGEN05 and info["kind"] == 2
    assert not (info["transposed"] and N % per)
    want, _ = oracle.gemm_reference(**p.oracle_args())
    want = torch.from_numpy(np.ascontiguousarray(want)).float().to(wl.TORCH_DTYPE[out]).double().numpy()
    np.testing.assert_array_equal(r.values(), want)
