"""Shared memory written by ordinary stores in both CTAs of a pair and read by the leader's tensor cores: the expanded
codes of the 8-bit product and the cleared rows of the weight gradient.  Every tile of a large call exact, again and
again; a store that the MMA overtook would show as a wrong integer."""
import numpy as np
import pytest
import torch

from test_gpu_grouped import BF16, F16, F32, run_wgrad
from test_gpu_i8 import run_i8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(3))
def test_expanded_codes(cuda_lib, seed):
    """33 tiles of 192 rows, and 110 ragged ones; 12 stages each, so every slot is filled many times."""
    for sizes, N in (([560], 2600), ([100, 0, 317, 64, 190, 1, 129], 2600)):
        got, want, _, path = run_i8(cuda_lib, sizes, N, 1500, F32, seed=seed, grouped=len(sizes) > 1)
        assert path == cuda_lib.PATH_TCGEN05
        np.testing.assert_array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("ab", [F16, BF16], ids=["f16", "bf16"])
def test_cleared_rows(cuda_lib, seed, ab):
    """Groups that end at every place of a k-block, 4 tiles each: 180 tiles for the 76 SM pairs."""
    sizes = np.random.default_rng(seed).integers(0, 200, size=45).tolist()
    for _ in range(4):
        got, want, _, path, sums = run_wgrad(cuda_lib, sizes, 300, 400, ab, F32, integer=True, seed=seed, first=3,
                                             after=9, poison=True)
        assert path == cuda_lib.PATH_TCGEN05
        np.testing.assert_array_equal(got, want)
        np.testing.assert_array_equal(sums[0], sums[1])


def test_same_bits_again(cuda_lib):
    g = cuda_lib
    gen = torch.Generator(device="cuda").manual_seed(1)
    M, N, K = 1000, 2600, 4100
    X = torch.randint(-128, 128, (M, 4112), dtype=torch.int8, device="cuda", generator=gen)
    W = torch.randint(-128, 128, (N, 4112), dtype=torch.int8, device="cuda", generator=gen)
    first = None
    for _ in range(20):
        C = torch.empty(M, N, device="cuda")
        g.gemm_i8(M, N, K, X, 4112, None, W, 4112, None, C, N, F32, 1.0, 0.0, None, 0)
        first = C if first is None else first
        assert torch.equal(C, first)
    assert g.gemm_device_status() == 0
