"""GPU tests of long sums in gemm_mx_grouped: fp32 sums, whatever the depth.

An instruction sums 32 E4M3 products onto the accumulator, and cuts the result off towards zero at 24 bits.  Rows here
have one product of 1 in instruction `big` and one of 1.5 * 2^-24 in each other one: beside a sum of 1 or more, whose
last place is 2^-23, each of these is cut off whole, so that an accumulator kept for the whole depth loses all that
follow `big` (191 units of 2^-23 at a depth of 8192).  Sums that are joined outside of it every 32 instructions lose at
most 31 of them, and half a unit at each joining: the bound, with nothing added.
"""
import numpy as np
import pytest
import torch

import oracle.mx_rows as om

pytestmark = pytest.mark.gpu

F32, F16, BF16 = 0, 1, 2
E4M3, E2M1 = 0, 1
SEGMENT = 32  # instructions


def padded(rows):
    """Rows of bytes at a pitch of whole 16."""
    return torch.from_numpy(np.pad(rows, ((0, 0), (0, -rows.shape[1] % 16))).astype(np.uint8)).cuda()


def coded(vals, scale_at, K):
    """E4M3 codes and scales of rows whose instruction i holds vals[:, i] * 2^scale_at[:, i] as its first product."""
    v = np.zeros((len(vals), K))
    v[:, ::32] = vals
    return padded(om.nearest_codes(v, E4M3)), padded(127 + scale_at)


@pytest.mark.parametrize("K", [512, 1024, 1056, 1184, 2080, 4096, 8192])
@pytest.mark.parametrize("rows", [5, 16, 33, 207, 208, 300])
def test_sums_do_not_lose_what_a_long_accumulator_would(cuda_lib, K, rows):
    g, N, n = cuda_lib, 272, K // 32
    big = np.arange(rows) * 7 % n
    x = np.where(np.arange(n) == big[:, None], 1.0, 1.5)
    X, XS = coded(x, np.where(x == 1.0, 0, -24), K)
    sign = np.where(np.arange(N) % 3 == 0, -1.0, 1.0)
    W, WS = coded(np.repeat(sign[:, None], n, 1), np.zeros((N, n), int), K)
    C = torch.full((rows + 1, N), 77.0, device="cuda")
    g.gemm_mx_grouped(1, rows, N, K, E4M3, None, X, X.shape[1], XS, XS.shape[1], W, 0, W.shape[1], WS, 0, WS.shape[1], C, N,
                      F32, 1.0, 0.0, None, 0)
    assert g.gemm_device_status() == 0 and (C[rows] == 77.0).all()
    want = (1 + (n - 1) * 1.5 * 2.0 ** -24) * sign
    bound = min(n - 1, SEGMENT - 1) * 1.5 * 2.0 ** -24 + (-(-n // SEGMENT) - 1) * 2.0 ** -24
    got = C[:rows].cpu().double().numpy()
    assert (np.abs(got - want) <= bound).all(), f"off by {np.abs(got - want).max() * 2 ** 23:.2f} units of 2^-23"


def test_4_bit_sums_are_exact_below_24_bits(cuda_lib):
    """One sign, 8192 deep, scales up to four powers of two apart (two in each operand): below 2^24 of the smallest
    product, exact."""
    g, M, N, K = cuda_lib, 219, 270, 8192
    rng = np.random.default_rng(0)
    codes = [rng.integers(0, 8, (r, K)) for r in (M, N)]
    scales = [rng.integers(127, 130, (r, K // 32)) for r in (M, N)]
    xv, wv = (om.values_of(c, s, E2M1) for c, s in zip(codes, scales))
    X, W = (padded(om.packed(c, E2M1)) for c in codes)
    XS, WS = (padded(s) for s in scales)
    C = torch.empty(M, N, device="cuda")
    g.gemm_mx_grouped(1, M, N, K, E2M1, None, X, K, XS, K // 32, W, 0, K, WS, 0, K // 32, C, N, F32, 1.0, 0.0, None, 0)
    want = xv @ wv.T
    assert want.max() * 4 < 2 ** 24
    np.testing.assert_array_equal(C.cpu().double().numpy(), want)


@pytest.mark.parametrize("elem", [E4M3, E2M1], ids=["e4m3", "e2m1"])
@pytest.mark.parametrize("out", [F32, F16, BF16])
def test_deep_sums_of_integers_in_ragged_groups(cuda_lib, elem, out):
    """Several joinings a tile, many tiles a pair of SMs, widths of every half, bias and beta: whole numbers, exact
    (below 2^24 in fp32; at most 2^11 and 2^8 in 16 bits, of thin rows)."""
    g, N, K = cuda_lib, 600, 4128
    rng = np.random.default_rng(out)
    sizes = [0, 1, 16, 17, 31, 33, 0, 47, 48, 80, 111, 112, 113, 176, 195, 207, 208, 209, 430, 3]
    off = np.concatenate([[0], np.cumsum(sizes)])
    M, G = int(off[-1]), len(sizes)
    thin = 1.0 if out == F32 else {F16: 0.02, BF16: 0.01}[out]

    def operand(rows, most):
        v = rng.integers(-most, most + 1, (rows, K)) * (rng.random((rows, K)) < thin)
        codes = om.packed(om.nearest_codes(v.astype(np.float64), elem), elem)
        s = np.full((rows, -(-(K // 32) // 16) * 16), 127, np.uint8)
        return v, torch.from_numpy(np.ascontiguousarray(np.pad(codes, ((0, 0), (0, -codes.shape[1] % 16))))).cuda(), \
            torch.from_numpy(s).cuda()

    xv, X, XS = operand(M, 2)
    wv, W, WS = operand(G * N, 1 if out == BF16 else 2)
    per, dt = {E4M3: 1, E2M1: 2}[elem], {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}[out]
    c0 = torch.from_numpy(rng.integers(-3, 4, (M, N))).to(dt)
    bias = torch.from_numpy(rng.integers(-3, 4, (G, N))).float()
    C = c0.cuda()
    g.gemm_mx_grouped(G, M, N, K, elem, torch.from_numpy(off).int().cuda(), X, X.shape[1] * per, XS, XS.shape[1], W,
                      N * W.shape[1] * per, W.shape[1] * per, WS, N * WS.shape[1], WS.shape[1], C, N, out, 1.0, 1.0,
                      bias.cuda(), g.EPI_BIAS)
    want = c0.double().numpy() + np.repeat(bias.double().numpy(), sizes, 0)
    for e in range(G):
        r = slice(off[e], off[e + 1])
        want[r] += xv[r] @ wv.reshape(G, N, K)[e].T
    assert np.abs(want).max() <= {F32: 2 ** 24, F16: 2 ** 11, BF16: 2 ** 8}[out]
    np.testing.assert_array_equal(C.cpu().double().numpy(), want)
