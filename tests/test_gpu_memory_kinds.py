"""GPU tests of the ranges that calls check: each kind of memory a kernel can read, and what lies past its end.

The arrays that reach past an allocation are never read: the rows' sources name none, and the groups have no rows.
"""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = 0, 2
N = 3000 * 64  # values of 4 bytes


@pytest.fixture(scope="module")
def runtime(cuda_lib):
    torch.zeros(1, device="cuda")
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libcudart" in line}
    return ctypes.CDLL(sorted(paths)[0])


@pytest.fixture(params=["device", "managed", "pinned", "registered", "registered inside a page"])
def memory(request, runtime):
    """An address and its bytes, freed afterwards; only what was allocated (or registered) counts."""
    p, kind, nbytes = ctypes.c_void_p(), request.param, 4 * N
    if kind.startswith("registered"):
        buf = np.zeros(nbytes + (1 << 17), np.uint8)
        at = (buf.ctypes.data + 65535) // 65536 * 65536 + (256 if "inside" in kind else 0)
        assert runtime.cudaHostRegister(ctypes.c_void_p(at), ctypes.c_size_t(nbytes), 0) == 0
        yield at, nbytes
        torch.cuda.synchronize()
        assert runtime.cudaHostUnregister(ctypes.c_void_p(at)) == 0
        return
    made = {"device": lambda: runtime.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(nbytes)),
            "managed": lambda: runtime.cudaMallocManaged(ctypes.byref(p), ctypes.c_size_t(nbytes), 1),
            "pinned": lambda: runtime.cudaHostAlloc(ctypes.byref(p), ctypes.c_size_t(nbytes), 3)}[kind]()
    assert made == 0
    yield p.value, nbytes
    torch.cuda.synchronize()
    assert (runtime.cudaFreeHost if kind == "pinned" else runtime.cudaFree)(p) == 0


def gather(g, x, rows, ldx, source):
    out = torch.full((source.numel(), 64), -1.0, device="cuda")
    g.gemm_rows_gather(source.numel(), 64, rows, 1, F32, x, ldx, source, None, out, 64)
    torch.cuda.synchronize()
    return out


def grouped(g, a, rows):
    """gemm_grouped of `rows` rows of 64 bf16, none of them in the group."""
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    w, c = (torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda") for n in (64, rows))
    g.gemm_grouped(1, rows, 64, 64, BF16, off, a, 64, 1, w, 4096, 1, 64, c, 64, BF16, 1.0, 0.0, None, 0)
    torch.cuda.synchronize()


def test_rows_in_every_kind_of_memory(cuda_lib, memory):
    """Read where they are; refused from the first byte past the end, whichever call asks."""
    g, (p, nbytes) = cuda_lib, memory
    values = torch.arange(N, dtype=torch.float32)
    fill = torch.empty(N, device="cuda").copy_(values)
    g.gemm_rows_gather(3000, 64, 3000, 1, F32, fill, 64, torch.arange(3000, dtype=torch.int32, device="cuda"), None, p, 64)
    source = torch.tensor([0, 2999, 17], dtype=torch.int32, device="cuda")
    assert torch.equal(gather(g, p, 3000, 64, source).cpu(), values.view(3000, 64)[[0, 2999, 17]])
    none = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    assert (gather(g, p + 4 * 64, 2999, 64, none) == -1).all()
    grouped(g, p, nbytes // 128)
    for x, rows, ldx in ((p, 3001, 64), (p + 256, 3000, 64), (p, 3000, 65), (p + nbytes - 252, 1, 64)):
        with pytest.raises(g.GemmError) as e:
            gather(g, x, rows, ldx, none)
        assert e.value.status == 1
    with pytest.raises(g.GemmError) as e:
        grouped(g, p, nbytes // 128 + 1)
    assert e.value.status == 1


def test_pageable_memory_is_refused(cuda_lib, runtime):
    g, buf = cuda_lib, np.zeros(N, np.float32)
    none = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(g.GemmError) as e:
        gather(g, buf.ctypes.data // 64 * 64 + 64, 100, 64, none)
    assert e.value.status == 1
    with pytest.raises(g.GemmError) as e:
        grouped(g, buf.ctypes.data // 64 * 64 + 64, 100)
    assert e.value.status == 1
