"""Long sums of the grouped products against float64.

The tensor cores add 16 products to an fp32 sum at a time and cut off what falls below its last place: less than
2^-23 of the sum, always towards zero, so on one-sided values the losses add up.  The kernels therefore add what 512
terms gave (32 such additions, at most 32 * 2^-23 = 2^-18 of them) into a separate fp32 sum, rounded to nearest (at
most 2^-24 of the sum per addition).  All inputs are positive here, so the sum itself is the scale:

    |got - want| <= (2^-18 + pieces * 2^-24) * sum + u * |want|,   pieces = terms / 512 + 8

(8: the partial sums that the kernel for few rows joins; u: the output's unit roundoff).  Without the pieces 16384
terms lose about 16384 / 16 * 2^-23 / 4 = 3e-5 of the sum, five times the bound.  16-bit outputs would round that
away, so they are asked for sum - C with C the rounded sum itself: what is left is small and shows it.
"""
import numpy as np
import pytest
import torch

from test_gpu_grouped import BF16, DT, F16, F32, NAMES, ROUNDOFF, offsets_of

pytestmark = pytest.mark.gpu


def positive(rng, shape, dt):
    t = torch.from_numpy(rng.uniform(0.25, 0.75, size=shape)).to(DT[dt])
    return t.cuda(), t.double().numpy()


def output(want, out):
    """C before the call (the rounded sums, or NaN that must not be read), beta, and the exact result."""
    if out == F32:
        return torch.full(want.shape, float("nan"), device="cuda"), 0.0, want
    C = torch.from_numpy(want).to(DT[out])
    return C.cuda(), -1.0, want - C.double().numpy()


def check(got, want, total, terms, out):
    bound = (2.0 ** -18 + (terms / 512 + 8) * 2.0 ** -24) * total + ROUNDOFF[out] * np.abs(want)
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= bound).all(), f"{np.nanmax(err / np.maximum(bound, 1e-300)):.2f} of the bound"


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_pair_kernel(cuda_lib, ab, out):
    g = cuda_lib
    rng = np.random.default_rng(ab)
    sizes, N, K = [33, 0, 70], 104, 16384
    G, M = len(sizes), sum(sizes)
    off = offsets_of(sizes)
    A, Av = positive(rng, (M, K), ab)
    B, Bv = positive(rng, (G, K, N), ab)
    total = np.concatenate([Av[off[e]:off[e + 1]] @ Bv[e] for e in range(G)])
    C, beta, want = output(total, out)
    g.gemm_grouped(G, M, N, K, ab, torch.from_numpy(off).int().cuda(), A, K, 1, B, K * N, N, 1, C, N, out, 1.0, beta,
                   None, 0)
    assert g.gemm_last_launch()["path"] == g.PATH_TCGEN05 and g.gemm_device_status() == 0
    check(C, want, total, K, out)


@pytest.mark.parametrize("rows", [1, 12, 30])
@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_few_rows(cuda_lib, ab, out, rows):
    """Each warp of that kernel sums an eighth of k (a quarter from 17 rows on)."""
    g = cuda_lib
    rng = np.random.default_rng(rows)
    N, K = 40, 131072
    A, Av = positive(rng, (rows, K), ab)
    B, Bv = positive(rng, (N, K), ab)
    total = Av @ Bv.T
    C, beta, want = output(total, out)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    g.gemm_grouped(1, rows, N, K, ab, off, A, K, 1, B, N * K, 1, K, C, N, out, 1.0, beta, None, 0)
    assert g.gemm_last_launch()["path"] == g.PATH_SIMT and g.gemm_device_status() == 0
    check(C, want, total, K, out)


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_weight_gradient(cuda_lib, ab, out):
    g = cuda_lib
    rng = np.random.default_rng(ab)
    sizes, M, N = [700, 16384, 0, 9001], 72, 104
    G, T = len(sizes), sum(sizes)
    off = offsets_of(sizes)
    A, Av = positive(rng, (T, M), ab)
    D, Dv = positive(rng, (T, N), ab)
    total = np.stack([Av[off[e]:off[e + 1]].T @ Dv[off[e]:off[e + 1]] for e in range(G)])
    C, beta, want = output(total, out)
    g.gemm_grouped_wgrad(G, T, M, N, ab, torch.from_numpy(off).int().cuda(), A, M, 1, D, N, 1, C, M * N, N, out, 1.0,
                         beta)
    assert g.gemm_last_launch()["path"] == g.PATH_TCGEN05 and g.gemm_device_status() == 0
    check(C, want, total, max(sizes), out)
