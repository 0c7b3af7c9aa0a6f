"""An 8-bit product's outputs do not depend on how many rows the call has or on which kernel runs it: the integer sum is
exact and every kernel rounds in the same places.  The first rows of calls of several sizes, aligned and not, bit for
bit equal, with an alpha that is no power of two, random scales, beta, bias and every activation."""
import numpy as np
import pytest
import torch

from test_gpu_grouped import BF16, DT, F16, F32, NAMES

pytestmark = pytest.mark.gpu

N, K, ROWS = 2600, 1031, 200  # 200 rows fill the pair kernel; 3, 8, 16 and 32 take the other forms


@pytest.fixture(scope="module")
def data(cuda_lib):
    rng = np.random.default_rng(11)
    X, W = (torch.from_numpy(rng.integers(-128, 128, size=(r, K)).astype(np.int8)) for r in (ROWS, N))
    f = [torch.from_numpy(np.float32(v)).cuda() for v in (rng.uniform(0.01, 0.05, ROWS), rng.uniform(0.01, 0.05, N) / 8,
                                                          rng.standard_normal(N), rng.standard_normal((ROWS, N)))]

    def pitch(t, ld):
        p = torch.zeros(t.shape[0], ld, dtype=torch.int8)
        p[:, :K] = t
        return p.cuda()

    return {ld: (pitch(X, ld), pitch(W, ld)) for ld in (1040, 1033)}, f


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("epi", range(6))
@pytest.mark.parametrize("beta", [0.0, 0.7])
@pytest.mark.parametrize("row_scale", [True, False], ids=["rs", "no_rs"])
def test_every_kernel_gives_the_same_bits(cuda_lib, data, out, epi, beta, row_scale):
    g = cuda_lib
    operands, (xs, ws, bias, C0) = data
    first = None
    for ld, (X, W) in operands.items():
        for M in (ROWS, 32, 16, 8, 3):
            C = C0[:M].to(DT[out], copy=True)
            g.gemm_i8(M, N, K, X, ld, xs if row_scale else None, W, ld, ws, C, N, out, 0.3, beta,
                      bias if epi else None, epi)
            assert (g.gemm_last_launch()["path"] == g.PATH_TCGEN05) == (ld == 1040 and M == ROWS)
            if first is None:
                first = C
            assert torch.equal(C, first[:M]), (ld, M, int((C != first[:M]).sum()))
    assert g.gemm_device_status() == 0 and bool(torch.isfinite(first).all())
