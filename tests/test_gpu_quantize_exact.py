"""gemm_i8_quantize's codes are round_even of the exact quotient for every input type: values on ties and one unit in
the last place beside them, from ordinary, tiny (subnormal) and huge rows, through each of its kernels."""
import numpy as np
import pytest
import torch

from oracle import grouped as og
from test_gpu_grouped import BF16, DT, F16, F32, NAMES

pytestmark = pytest.mark.gpu


def near_ties(rng, rows, K, dt):
    """(n + 1/2) max / 127 for random n, rounded to the type, and its neighbours; the maximum somewhere in the row.
    (The float64 reference is exact: 127 x has 31 bits, and a quotient that is no tie is 2^-33 from one.)"""
    lo = {F32: 1 << 23, F16: 1 << 10, BF16: 1 << 7}[dt]
    peak = torch.from_numpy(rng.integers(lo, 2 * lo, size=(rows, 1)).astype(np.float64)) / lo
    n = torch.from_numpy(rng.integers(0, 127, size=(rows, K)).astype(np.float64))
    x = ((n + 0.5) * peak / 127).to(DT[dt]).double()
    ulp = 2.0 ** torch.floor(torch.log2(x)) / lo
    x = x + ulp * torch.from_numpy(rng.integers(-1, 2, size=(rows, K)).astype(np.float64))
    x = torch.minimum(x, peak) * torch.from_numpy(rng.choice([-1.0, 1.0], size=(rows, K)))
    x[torch.arange(rows), torch.from_numpy(rng.integers(0, K, size=rows))] = peak[:, 0]
    return x


def quantize(g, t, pad, shift):
    """Codes and scales of t with rows `pad` longer, from a base `shift` elements past an aligned one."""
    M, K = t.shape
    ld = K + pad
    buf = torch.zeros(shift + M * ld, dtype=t.dtype)
    buf[shift:].view(M, ld)[:, :K] = t
    buf = buf.cuda()
    q = torch.full((M, ld), 55, dtype=torch.int8, device="cuda")
    s = torch.empty(M, device="cuda")
    g.gemm_i8_quantize(M, K, {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}[t.dtype],
                       buf.data_ptr() + shift * buf.element_size(), ld, q, ld, s)
    assert g.gemm_device_status() == 0 and bool((q[:, K:] == 55).all())
    return q[:, :K].cpu().numpy(), s.cpu().numpy()


def check(g, t, pad=0, shift=0):
    want_q, want_s = og.quantize_reference(t.double().numpy())
    q, s = quantize(g, t, pad, shift)
    np.testing.assert_array_equal(q, want_q)
    np.testing.assert_array_equal(s, want_s.astype(np.float32))


@pytest.mark.parametrize("dt", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("K", [1000, 1001, 4096])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (0, 1)])
def test_ties_and_their_neighbours(cuda_lib, dt, K, pad, shift):
    check(cuda_lib, near_ties(np.random.default_rng(K + pad), 40, K, dt).to(DT[dt]), pad, shift)


@pytest.mark.parametrize("dt,exponents", [(F32, (-149, -140, -127, -101, -99, 99, 101, 127)), (F16, (-14, 4, 15)),
                                          (BF16, (-133, -128, -101, -99, 99, 101, 127))], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [1000, 1003])
def test_tiny_and_huge_rows(cuda_lib, dt, exponents, K):
    x = near_ties(np.random.default_rng(K), len(exponents) * 4, K, dt)
    x = x * (2.0 ** torch.tensor(exponents, dtype=torch.float64)).repeat_interleave(4)[:, None]
    top = float(torch.finfo(DT[dt]).max)
    check(cuda_lib, x.clamp(-top, top).to(DT[dt]))


@pytest.mark.parametrize("dt", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("pieces", [20, 130, 300, 700, 1500])
def test_many_rows(cuda_lib, dt, pieces):
    """Enough rows for the kernel that fetches ahead, with 1, 2, 4 and 8 pieces of 16 bytes per thread: the counts
    are odd ones, so that the last warps hold part of a row.  (At most 64 values of a row are next to ties.)"""
    rng = np.random.default_rng(pieces)
    K = pieces * (4 if dt == F32 else 8)
    rows = 2600 if pieces > 200 else 12000
    gen = torch.Generator().manual_seed(pieces)
    t = torch.randn(rows, K, generator=gen).to(DT[dt])
    t[::7, :64] = near_ties(rng, len(t[::7]), 64, dt).to(DT[dt]) * 4  # some maxima there, others among the rest
    t[5] = 0
    t[11, K - 1] = float("nan")
    t[rows - 1, 0] = float("-inf")
    check(cuda_lib, t)
