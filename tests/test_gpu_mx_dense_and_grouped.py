"""GPU test of the two block-scaled products against each other: gemm_mx and gemm_mx_grouped read the same codes and
scales, so whole numbers, whose sums are exact, come out the same bits (order of scales, nibbles and rows alike)."""
import numpy as np
import pytest
import torch

import oracle.mx_rows as om

pytestmark = pytest.mark.gpu

F32, F16, BF16 = 0, 1, 2
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
E4M3, E2M1 = 0, 1


@pytest.mark.parametrize("elem", [E4M3, E2M1], ids=["e4m3", "e2m1"])
@pytest.mark.parametrize("M,N,K", [(333, 520, 512), (1, 256, 1024), (700, 264, 4096)])
@pytest.mark.parametrize("out", [F32, F16, BF16])
@pytest.mark.parametrize("grouped", [False, True], ids=["rows", "offsets"])
def test_one_group_is_the_dense_product(cuda_lib, elem, M, N, K, out, grouped):
    g = cuda_lib
    rng = np.random.default_rng(M + K)
    per, blocks = {E4M3: 1, E2M1: 2}[elem], K // 32

    def operand(rows):
        v = rng.integers(-2, 3, (rows, K)).astype(np.float64)
        s = rng.integers(127, 129, (rows, blocks)).astype(np.uint8)
        return torch.from_numpy(om.packed(om.nearest_codes(v, elem), elem)).cuda(), torch.from_numpy(s).cuda(), \
            v * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, 1)

    X, XS, xv = operand(M)
    W, WS, wv = operand(N)
    want = xv @ wv.T
    assert np.abs(want).max() < 2 ** 24
    alpha = 1.0 if out == F32 else 2.0 ** -9
    dense, one = (torch.full((M, N), float("nan"), dtype=DT[out], device="cuda") for _ in range(2))
    ws = torch.empty(max(16, g.gemm_mx_workspace_size(M, N, K, elem)), dtype=torch.uint8, device="cuda")
    g.gemm_mx(M, N, K, elem, X, K, XS, W, K, WS, dense, N, out, alpha, 0.0, None, g.EPI_NONE, ws, ws.numel())
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda") if grouped else None
    g.gemm_mx_grouped(1, M, N, K, elem, offsets, X, K, XS, blocks, W, 0, K, WS, 0, blocks, one, N, out, alpha, 0.0, None,
                      g.EPI_NONE)
    assert g.gemm_device_status() == 0
    assert torch.equal(dense, one)
    assert torch.equal(one, torch.from_numpy(want * alpha).float().to(DT[out]).cuda())
