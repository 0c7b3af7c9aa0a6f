"""Offsets that break their rules: no access leaves the arrays, no row is computed twice, every row that is written
holds what one of the groups gives it.  (The first two would show as a fault or a race, so these run on kernels whose
group table has been read to hold them.)"""
import pytest
import torch

from test_gpu_grouped import BF16, CANARY, F16, F32

pytestmark = pytest.mark.gpu


def bias_rows(g, M, N, offsets, K=0):
    """C rows = the number of the group that wrote them (1-based), CANARY where none did."""
    G = len(offsets) - 1
    bias = torch.arange(1, G + 1, device="cuda", dtype=torch.float32)[:, None].expand(G, N).contiguous()
    C = torch.full((M + 8, N), CANARY, device="cuda")
    A = torch.zeros(M, max(K, 8), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(G, N, max(K, 8), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int64).to(torch.int32).cuda()
    g.gemm_grouped(G, M, N, K, BF16, off, A, max(K, 8), 1, B, N * max(K, 8), 1, max(K, 8), C, N, F32, 1.0, 0.0, bias,
                   g.EPI_BIAS)
    assert g.gemm_device_status() == 0
    assert bool((C[M:] == CANARY).all())
    assert bool((C == C[:, :1]).all())
    return C[:M, 0].tolist()


@pytest.mark.parametrize("N,K", [(8, 0), (40, 64), (4096, 64)], ids=["cuda_cores", "few_rows", "pair"])
def test_each_row_has_one_group(cuda_lib, N, K):
    got = bias_rows(cuda_lib, 100, N, [0, 50, 20, 100], K)
    assert got == [1.0] * 50 + [3.0] * 50  # the second group ends at 50 too, the third begins there
    got = bias_rows(cuda_lib, 600, N, [500, 20, 10, 590, 580, 600, 0], K)
    assert got[:500] == [CANARY] * 500 and got[500:590] == [3.0] * 90 and got[590:] == [5.0] * 10
    got = bias_rows(cuda_lib, 300, N, [-(1 << 31), (1 << 31) - 1, -5, 300], K)
    assert got == [1.0] * 300


def test_row_tiles_of_overlapping_groups_stay_in_32_bits(cuda_lib):
    """512 groups that would each be all of 2^31 - 1024 rows: together 2^34 tiles of 64 rows."""
    g = cuda_lib
    M, G = g.GROUPED_MAX_EXTENT, 1024
    C = torch.zeros(M + 64, dtype=torch.float16, device="cuda")
    C[M:] = CANARY
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[1::2] = M
    bias = torch.full((G, 1), 9.0, device="cuda")
    bias[0] = 3.0
    g.gemm_grouped(G, M, 1, 0, F16, off, None, 0, 0, None, 0, 0, 0, C, 1, F16, 1.0, 0.0, bias, g.EPI_BIAS)
    assert g.gemm_device_status() == 0
    assert bool((C[:M] == 3.0).all()) and bool((C[M:] == CANARY).all())
