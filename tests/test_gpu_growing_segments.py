"""GPU test of tensors in virtual memory that is mapped in pieces (PyTorch's growing segments): taken by every call as
other device memory is, refused where nothing is mapped.  In a process of its own, since an allocator is chosen once."""
import os
import subprocess
import sys

import pytest

from conftest import REPO

pytestmark = pytest.mark.gpu

PROGRAM = """
import os
for name in ("PYTORCH_ALLOC_CONF", "PYTORCH_CUDA_ALLOC_CONF"):
    os.environ[name] = "expandable_segments:True"
import torch
import dense_gemm_epilogues_tcgen05_gb300 as g

def bits(rows, n):  # small integers, so that sums are exact
    return torch.randint(-2, 3, (rows, n), device="cuda", dtype=torch.int8).bfloat16()

n = 1024
w = torch.eye(n, device="cuda").bfloat16()
for rows in (100, 60000):
    x, c = bits(rows, n), torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    need = max(16, g.gemm_workspace_size(rows, n, n, g.BF16))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    g.gemm(rows, n, n, g.BF16, x, n, 1, w, 1, n, c, n, g.BF16, 1.0, 0.0, None, g.EPI_NONE, ws, need)
    assert torch.equal(c, x)
    c.zero_()
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    g.gemm_grouped(1, rows, n, n, g.BF16, off, x, n, 1, w, 0, 1, n, c, n, g.BF16, 1.0, 0.0, None, g.EPI_NONE)
    assert torch.equal(c, x)
    c.zero_()
    source = torch.arange(rows, dtype=torch.int32, device="cuda").flip(0).contiguous()
    g.gemm_rows_gather(rows, n, rows, 1, g.BF16, x, n, source, None, c, n)
    assert torch.equal(c, x.flip(0))
    assert g.gemm_device_status() == 0
# rows that no source names, past what is mapped: refused, and so is a group of no rows there
none = torch.full((4,), -1, dtype=torch.int32, device="cuda")
out = torch.zeros(4, n, dtype=torch.bfloat16, device="cuda")
empty = torch.zeros(2, dtype=torch.int32, device="cuda")
far = 1 << 24  # 32 GB of rows
for call in (lambda: g.gemm_rows_gather(4, n, far, 1, g.BF16, x, n, none, None, out, n),
             lambda: g.gemm_grouped(1, 4, n, n, g.BF16, empty, x, far * n, 1, w, 0, 1, n, out, n, g.BF16, 1.0, 0.0, None, 0)):
    try:
        call()
    except g.GemmError as e:
        assert e.status == g.ERR_INVALID_ARG
    else:
        raise SystemExit("taken")
torch.cuda.synchronize()
print("all of them")
"""


def test_tensors_in_growing_segments(cuda_lib):
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300, cwd=REPO,
                       env=dict(os.environ, PYTHONPATH=REPO))
    assert r.returncode == 0 and "all of them" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
