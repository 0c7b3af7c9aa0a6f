"""GPU tests of the 8-bit integer products (gemm_i8, gemm_i8_grouped) and gemm_i8_quantize.

The integer sum is exact, so with power-of-two scales and fp32 output every result is one rounding of an
exact value: bit for bit what numpy's float32 gives from int64 sums, for codes that reach far beyond 2^24.
Quantised codes of 16-bit inputs equal the exact quotient's rounding.
"""
import numpy as np
import pytest
import torch

from oracle import grouped as og
from test_gpu_grouped import BF16, CANARY, DT, F16, F32, NAMES, SPLITS, check, offsets_of

pytestmark = pytest.mark.gpu


def codes(rng, shape, kind):
    if kind == "extreme":  # every product 128 * 128: the largest sums there are
        return np.full(shape, -128, dtype=np.int8)
    if kind == "positive":  # one-sided: sums far past 2^24
        return rng.integers(90, 128, size=shape).astype(np.int8)
    return rng.integers(-128, 128, size=shape).astype(np.int8)


def padded(a, ld, fill=-99):
    p = np.full((*a.shape[:-1], ld), fill, dtype=np.int8)
    p[..., :a.shape[-1]] = a
    return torch.from_numpy(p).cuda()


def run_i8(g, sizes, N, K, out, *, seed=0, kind="any", epi=0, alpha=1.0, beta=0.0, scales="pow2", grouped=True,
           align=16, ldc_pad=3, first=0, after=0):
    rng = np.random.default_rng(seed)
    G, off = len(sizes), offsets_of(sizes, first)
    M = int(off[-1]) + after
    X, W = codes(rng, (M, K), kind), codes(rng, (G, N, K), kind)
    ld = (K + align - 1) // align * align + align
    xs = ws = None
    if scales == "pow2":
        xs, ws = 2.0 ** rng.integers(-3, 4, size=M), 2.0 ** rng.integers(-3, 4, size=(G, N))
    elif scales == "random":
        xs, ws = rng.uniform(0.01, 0.05, size=M), rng.uniform(0.01, 0.05, size=(G, N))
    xs, ws = (None if v is None else np.float32(v) for v in (xs, ws))
    C = torch.full((M + 2, N + ldc_pad), CANARY, dtype=DT[out])
    C0 = torch.from_numpy(rng.integers(-64, 65, size=(M, N)).astype(np.float64)).to(DT[out])
    C[1 + first:1 + int(off[-1]), :N] = C0[first:int(off[-1])] if beta != 0.0 else float("nan")
    before = C.clone()
    C = C.cuda()
    bias = np.float32(rng.integers(-64, 65, size=(G, N))) if epi else None
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    Xd, Wd = padded(X, ld), padded(W, ld)
    cp, ldc = C.data_ptr() + (N + ldc_pad) * C.element_size(), N + ldc_pad
    if grouped:
        g.gemm_i8_grouped(G, M, N, K, torch.from_numpy(off).int().cuda(), Xd, ld, dev(xs), Wd, N * ld, ld, dev(ws),
                          cp, ldc, out, alpha, beta, dev(bias), epi)
    else:
        g.gemm_i8(M, N, K, Xd, ld, dev(xs), Wd, ld, dev(ws), cp, ldc, out, alpha, beta, dev(bias), epi)
    path = g.gemm_last_launch()["path"]
    assert g.gemm_device_status() == 0
    C = C.cpu()
    keep = torch.ones(C.shape, dtype=torch.bool)
    keep[1 + first:1 + int(off[-1]), :N] = False
    assert torch.equal(C[keep], before[keep]), "wrote outside its rows"
    Y, D = og.grouped_reference(off, X.astype(np.float64), W.astype(np.float64).transpose(0, 2, 1), epi, alpha, beta,
                                C0.double().numpy() if beta else None, bias, xs, ws)
    sl = slice(first, int(off[-1]))
    return C[1:M + 1, :N].double().numpy()[sl], Y[sl], D[sl], path


# every row count around the boundaries of the kernels, then tile boundaries
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33, 65, 130, 200, 400])
@pytest.mark.parametrize("N,K", [(1, 16), (40, 100), (300, 1040), (129, 2500)], ids=str)
@pytest.mark.parametrize("kind", ["any", "positive"])
def test_exact_sums(cuda_lib, M, N, K, kind):
    got, want, _, _ = run_i8(cuda_lib, [M], N, K, F32, kind=kind, seed=M + N, grouped=False)
    np.testing.assert_array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("M", [1, 5, 12, 40, 300])
def test_largest_sums(cuda_lib, M):
    """K at its limit and every code -128: the sum 2147467264, one below what 32 bits hold."""
    K = cuda_lib.I8_MAX_K
    got, want, _, _ = run_i8(cuda_lib, [M], 20, K, F32, kind="extreme", grouped=False, scales="none")
    assert want[0, 0] == 16384.0 * K
    np.testing.assert_array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("split", SPLITS, ids=str)
@pytest.mark.parametrize("N,K", [(72, 48), (260, 1100)], ids=str)
def test_grouped_exact(cuda_lib, split, N, K):
    got, want, _, _ = run_i8(cuda_lib, SPLITS[split], N, K, F32, seed=K, first=2, after=3)
    np.testing.assert_array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("epi", range(6))
@pytest.mark.parametrize("sizes", [[3], [20], [150], [0, 33, 1, 90]], ids=str)
def test_epilogues(cuda_lib, out, epi, sizes):
    got, want, D, _ = run_i8(cuda_lib, sizes, 200, 333, out, epi=epi, alpha=0.25, beta=0.5, scales="random",
                             grouped=len(sizes) > 1)
    check(got, want, D, out)


@pytest.mark.parametrize("M", [1, 8, 20, 100])
@pytest.mark.parametrize("align", [1, 4, 16])
def test_alignment_gives_the_same_bits(cuda_lib, M, align):
    got, want, _, _ = run_i8(cuda_lib, [M], 77, 1031, F32, align=align, grouped=False, kind="positive")
    np.testing.assert_array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("ldc_pad", [0, 1, 2])
@pytest.mark.parametrize("M", [1, 6, 40])
@pytest.mark.parametrize("out", [F16, BF16], ids=NAMES.get)
def test_output_pitch(cuda_lib, ldc_pad, M, out):
    for N in (64, 99):
        got, want, D, _ = run_i8(cuda_lib, [M], N, 64, out, ldc_pad=ldc_pad, scales="random", grouped=False)
        check(got, want, D, out)


@pytest.mark.parametrize("M", [1, 40])
def test_no_product(cuda_lib, M):
    for K, alpha in ((0, 1.0), (64, 0.0)):
        got, want, D, path = run_i8(cuda_lib, [M], 33, K, F32, epi=4, alpha=alpha, beta=2.0, scales="random",
                                    grouped=False)
        check(got, want, D, F32)
        assert path == cuda_lib.PATH_EPILOGUE_ONLY


# ------------------------------------------------------------------ quantise --

@pytest.mark.parametrize("dt", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (3, 100), (5, 8192), (2, 40000), (37, 1003)], ids=str)
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_quantize(cuda_lib, dt, M, K, pad):
    g = cuda_lib
    rng = np.random.default_rng(K + M)
    x = rng.standard_normal((M, K)) * 10.0 ** rng.integers(-3, 3, size=(M, 1))
    if M > 1:
        x[1] = 0.0
    t = torch.full((M, K + pad), float("nan"), dtype=DT[dt])
    t[:, :K] = torch.from_numpy(x).to(DT[dt])
    q = torch.full((M, K + pad), 55, dtype=torch.int8, device="cuda")
    s = torch.full((M,), 9.0, device="cuda")
    g.gemm_i8_quantize(M, K, dt, t.cuda(), K + pad, q, K + pad, s)
    assert g.gemm_device_status() == 0
    want_q, want_s = og.quantize_reference(t[:, :K].double().numpy())
    q = q.cpu().numpy()
    assert (q[:, K:] == 55).all()
    off = np.abs(q[:, :K].astype(int) - want_q)
    if dt == F32:  # 127 x rounds: a quotient within 2^-16 of a tie may go either way
        assert off.max() <= 1 and (off > 0).mean() < 1e-3
    else:
        assert off.max() == 0
    np.testing.assert_array_equal(s.cpu().numpy(), want_s.astype(np.float32))


def test_quantize_ties_extremes_and_not_finite(cuda_lib):
    g = cuda_lib
    x = torch.zeros(6, 64, dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 127 * 2, 1, 3, -5  # quotients 127, .5, 1.5, -2.5: ties to even
    x[1, :] = float(torch.finfo(torch.bfloat16).max)
    x[1, 1] *= -1
    x[2, 5] = float("nan")
    x[3, 9] = float("-inf")
    x[4, 3] = 2.0 ** -130
    q = torch.empty(6, 64, dtype=torch.int8, device="cuda")
    s = torch.empty(6, device="cuda")
    g.gemm_i8_quantize(6, 64, BF16, x.cuda(), 64, q, 64, s)
    q, s = q.cpu(), s.cpu()
    assert q[0, :4].tolist() == [127, 0, 2, -2]
    assert q[1, 0] == 127 and q[1, 1] == -127 and (q[1, 2:] == 127).all()
    assert torch.isnan(s[2]) and torch.isnan(s[3]) and not q[2:4].any()
    assert q[4, 3] == 127 and s[4] == np.float32(2.0 ** -130 / 127)
    assert s[5] == 0 and not q[5].any()


@pytest.mark.parametrize("dt", [F16, BF16], ids=NAMES.get)
def test_quantize_near_ties(cuda_lib, dt):
    """Every mantissa of the type against many maxima: quotients on and next to ties, both signs."""
    g = cuda_lib
    bits = 11 if dt == F16 else 8
    mant = torch.arange(1 << (bits - 1), 1 << bits, dtype=torch.float64)
    x = torch.cat([mant, -mant / 2, mant / 4, -mant / 64]) / (1 << bits)  # all below 1
    rows = 64
    peaks = 1 + torch.arange(rows, dtype=torch.float64) / rows * (1 - 2.0 ** -7)
    t = torch.cat([x.expand(rows, -1), peaks[:, None]], 1).to(DT[dt])
    M, K = t.shape
    q = torch.empty(M, K, dtype=torch.int8, device="cuda")
    s = torch.empty(M, device="cuda")
    g.gemm_i8_quantize(M, K, dt, t.cuda(), K, q, K, s)
    padded_x = torch.zeros(M, K + 7, dtype=DT[dt])
    padded_x[:, :K] = t
    ld = (K + 7) // 8 * 8
    q2 = torch.empty(M, ld, dtype=torch.int8, device="cuda")
    g.gemm_i8_quantize(M, K, dt, padded_x[:, :ld].contiguous().cuda(), ld, q2, ld, s)  # the vector path
    want, _ = og.quantize_reference(t.double().numpy())
    np.testing.assert_array_equal(q.cpu().numpy(), want)
    np.testing.assert_array_equal(q2[:, :K].cpu().numpy(), want)


def test_quantize_then_multiply(cuda_lib):
    """The two together: x W^T of quantised x and W within half a step of each."""
    g = cuda_lib
    rng = np.random.default_rng(1)
    M, N, K = 19, 96, 512
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16)
    w = torch.from_numpy(rng.standard_normal((N, K))).to(torch.bfloat16)
    qx, qw = (torch.empty(t.shape, dtype=torch.int8, device="cuda") for t in (x, w))
    sx, sw = torch.empty(M, device="cuda"), torch.empty(N, device="cuda")
    g.gemm_i8_quantize(M, K, BF16, x.cuda(), K, qx, K, sx)
    g.gemm_i8_quantize(N, K, BF16, w.cuda(), K, qw, K, sw)
    y = torch.empty(M, N, device="cuda")
    g.gemm_i8(M, N, K, qx, K, sx, qw, K, sw, y, N, F32, 1.0, 0.0, None, 0)
    X, W = x.double(), w.double()
    ex, ew = sx.double().cpu() / 2, sw.double().cpu() / 2
    bound = ex[:, None] * W.abs().sum(1) + ew[None] * X.abs().sum(1)[:, None] + K * ex[:, None] * ew[None]
    assert ((y.cpu().double() - X @ W.T).abs() <= bound * (1 + 1e-5)).all()
