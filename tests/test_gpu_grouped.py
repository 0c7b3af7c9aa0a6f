"""GPU tests of the expert-grouped products (gemm_grouped, gemm_grouped_wgrad) against float64.

Integer-valued inputs whose partial sums stay below 2^24 come back bit-exact with fp32 output.  Random
inputs are held to |got - want| <= u |want| + 1e-5 D s: u the output type's unit roundoff (2^-24, 2^-11, 2^-8:
one rounding to nearest), 1e-5 of D the library's tolerance of an fp32 sum (D: the sum of absolute values
behind the output), s the activation's largest slope.  (2e-3 of D, the dense products' tolerance of 16-bit
outputs, is below a bf16 rounding where |want| = D, as for a group of one row.)  Gradients by differences are
exact by construction.  Rows and
columns outside the result keep their canary.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import grouped as og

pytestmark = pytest.mark.gpu

F32, F16, BF16 = 0, 1, 2
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
ROUNDOFF = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
CANARY = 77.0
NAMES = {F32: "f32", F16: "f16", BF16: "bf16"}

# group sizes: empty groups first, last and between; one row; a tile boundary; ragged
SPLITS = {
    "one": [5],
    "ragged": [0, 1, 33, 0, 130, 7, 0],
    "tiles": [256, 257, 255, 64],
    "many": [3] * 40 + [0] * 20 + [1] * 17,
    "empty": [0, 0, 0],
}


def offsets_of(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int64)


def values(rng, shape, integer):
    if integer:
        return rng.integers(-4, 5, size=shape).astype(np.float64)
    return rng.standard_normal(shape)


def to_dev(a, dt, ld=None, fill=float("nan")):
    """A device tensor of `a` rounded to dt, rows padded to pitch ld with `fill`; and the rounded values."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT[dt])
    back = t.double().numpy()
    if ld is not None and ld != a.shape[-1]:
        p = torch.full((*a.shape[:-1], ld), fill, dtype=DT[dt])
        p[..., :a.shape[-1]] = t
        t = p
    return t.cuda(), back


def check(got, want, D, out, slope=1.13):
    """The bound above, for every output; 2^-25 for an F16 output among the subnormals."""
    assert got.shape == want.shape
    bound = ROUNDOFF[out] * np.abs(want) + oracle.TOL_F32_OUT * slope * D + (2.0 ** -25 if out == F16 else 0.0)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst by {np.nanmax(np.abs(got - want) - bound):.3e}"


def run_grouped(g, sizes, N, K, ab, out, *, seed=0, integer=False, trans=False, epi=0, alpha=1.0, beta=0.0,
                row_scale=False, pad=0, first=0, after=0, ldc_pad=3, a_kmajor=True, stream=None, b_shift=0):
    """One call on guarded buffers; returns (result, reference, D, path)."""
    rng = np.random.default_rng(seed)
    G, off = len(sizes), offsets_of(sizes, first)
    M = int(off[-1]) + after
    ld = (K + 7) // 8 * 8 + pad
    if a_kmajor:
        A, Av = to_dev(values(rng, (M, K), integer), ab, ld)
        sam, sak = ld, 1
    else:
        lda = (M + 7) // 8 * 8
        At, Atv = to_dev(values(rng, (K, M), integer), ab, lda)
        A, Av, sam, sak = At, Atv.T, 1, lda
    Bv0 = values(rng, (G, K, N) if trans else (G, N, K), integer) * (1.0 if integer else 1 / np.sqrt(max(K, 1)))
    ldb = ((N if trans else K) + 7) // 8 * 8 + pad
    B, Bv = to_dev(Bv0, ab, ldb)
    if b_shift:  # the same weights from a base that TMA cannot read
        flat = torch.full((B.numel() + b_shift,), float("nan"), dtype=B.dtype, device="cuda")
        flat[b_shift:] = B.flatten()
        B = flat[b_shift:]
    sbg = Bv0.shape[1] * ldb
    sbk, sbn = (ldb, 1) if trans else (1, ldb)
    Bk = Bv if trans else Bv.transpose(0, 2, 1)
    ldc = N + ldc_pad
    C0 = values(rng, (M, N), integer)
    C = torch.full((M + 2, ldc), CANARY, dtype=DT[out])
    Cr = torch.from_numpy(C0).to(DT[out])
    if beta != 0.0:
        C[1:M + 1, :N] = Cr
    else:
        C[1 + first:1 + int(off[-1]), :N] = float("nan")  # beta == 0 must not read C
    before = C.clone()
    C = C.cuda()
    bias = torch.from_numpy(values(rng, (G, N), integer)).float() if epi else None
    rs = torch.from_numpy(rng.choice([0.5, 1.0, 2.0], size=M)).float() if row_scale else None
    g.gemm_grouped(G, M, N, K, ab, torch.from_numpy(off).int().cuda(), A, sam, sak, B, sbg, sbk, sbn,
                   C.data_ptr() + ldc * C.element_size(), ldc, out, alpha, beta, None if bias is None else bias.cuda(),
                   epi, row_scale=None if rs is None else rs.cuda(), stream=stream)
    path = g.gemm_last_launch()["path"]
    assert g.gemm_device_status(stream) == 0
    C = C.cpu()
    keep = np.ones(C.shape, dtype=bool)
    keep[1 + first:1 + int(off[-1]), :N] = False
    assert torch.equal(C[torch.from_numpy(keep)], before[torch.from_numpy(keep)]), "wrote outside its rows"
    Y, D = og.grouped_reference(off, Av, Bk, epi, alpha, beta, Cr.double().numpy() if beta else None,
                                None if bias is None else bias.double().numpy(),
                                None if rs is None else rs.double().numpy())
    sl = slice(first, int(off[-1]))
    return C[1:M + 1, :N].double().numpy()[sl], Y[sl], D[sl], path


@pytest.mark.parametrize("split", SPLITS, ids=str)
@pytest.mark.parametrize("N,K", [(1, 8), (72, 64), (300, 200), (257, 1000)], ids=str)
@pytest.mark.parametrize("trans", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_integer_exact(cuda_lib, split, N, K, trans, ab):
    """Exact sums: a wrong row, column, group, k tail or accumulator shows as a wrong integer."""
    got, want, _, path = run_grouped(cuda_lib, SPLITS[split], N, K, ab, F32, integer=True, trans=trans,
                                     seed=N + K, pad=8, first=3, after=5)
    assert path in (cuda_lib.PATH_TCGEN05, cuda_lib.PATH_SIMT)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("split", ["ragged", "tiles", "many"])
@pytest.mark.parametrize("N,K", [(1500, 72), (1513, 840)], ids=str)
@pytest.mark.parametrize("trans", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("out", [F32, BF16], ids=NAMES.get)
def test_integer_exact_on_the_pair_kernel(cuda_lib, split, N, K, trans, out):
    """Enough column tiles that no call takes the kernel for few rows; bf16 outputs are the rounded sums."""
    got, want, _, path = run_grouped(cuda_lib, SPLITS[split], N, K, BF16, out, integer=True, trans=trans, seed=N + K,
                                     first=3, after=5, ldc_pad=4 - N % 4)
    assert path == cuda_lib.PATH_TCGEN05
    if out == BF16:
        want = torch.from_numpy(want).bfloat16().double().numpy()
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("N,K", [(1, 64), (33, 8), (200, 1000), (517, 4160)], ids=str)
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_few_rows(cuda_lib, rows, N, K, ab):
    """One group, and the rows split unevenly over three."""
    for sizes in ([rows], [rows // 2, 0, rows - rows // 2]):
        got, want, _, _ = run_grouped(cuda_lib, sizes, N, K, ab, F32, integer=True, seed=rows + N, first=1, after=2)
        np.testing.assert_array_equal(got, want)
    got, want, D, _ = run_grouped(cuda_lib, [rows], N, K, ab, ab, epi=4, alpha=0.5, beta=0.25, row_scale=True, seed=K)
    check(got, want, D, ab)


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("epi", range(6))
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_epilogues(cuda_lib, epi, out, ab):
    """Every epilogue and output type with alpha, beta * C and the row scale."""
    got, want, D, _ = run_grouped(cuda_lib, SPLITS["ragged"], 200, 328, ab, out, epi=epi, alpha=0.75, beta=0.5,
                                  row_scale=True, seed=epi)
    check(got, want, D, out)


@pytest.mark.parametrize("ldc_pad", [0, 1, 2, 5])
@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
def test_output_pitch(cuda_lib, ldc_pad, out):
    """Row pitches that rule out pairs or 16-byte vectors, N odd and even."""
    for N in (64, 99):
        got, want, D, _ = run_grouped(cuda_lib, [70, 0, 41], N, 72, BF16, out, ldc_pad=ldc_pad, integer=True)
        if out == BF16:
            want = torch.from_numpy(want).bfloat16().double().numpy()
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("sizes", [[900, 30, 2000], [128] * 9], ids=str)
def test_random_large(cuda_lib, sizes):
    got, want, D, _ = run_grouped(cuda_lib, sizes, 768, 2048, BF16, BF16, seed=5)
    check(got, want, D, BF16)


def test_fp32_inputs_run(cuda_lib):
    got, want, D, path = run_grouped(cuda_lib, SPLITS["ragged"], 45, 77, F32, F32, epi=2, row_scale=True)
    check(got, want, D, F32)
    assert path == cuda_lib.PATH_SIMT


@pytest.mark.parametrize("kw", [dict(a_kmajor=False), dict(pad=3), dict(b_shift=1)], ids=str)
def test_strides_tma_cannot_read(cuda_lib, kw):
    got, want, D, path = run_grouped(cuda_lib, SPLITS["ragged"], 90, 100, F16, F32, integer=True, **kw)
    np.testing.assert_array_equal(got, want)
    assert path == cuda_lib.PATH_SIMT


@pytest.mark.parametrize("K,alpha", [(0, 1.0), (64, 0.0)])
def test_no_product(cuda_lib, K, alpha):
    """K == 0 or alpha == 0: act(beta C + bias), inputs and scales unread."""
    got, want, D, path = run_grouped(cuda_lib, SPLITS["ragged"], 33, K, BF16, F32, epi=4, alpha=alpha, beta=2.0,
                                     row_scale=True)
    check(got, want, D, F32)
    assert path == cuda_lib.PATH_EPILOGUE_ONLY


def test_not_finite_stays_in_its_rows(cuda_lib):
    """Infinities and NaN of one group reach that group's rows alone, next to tiles that share its loads."""
    g = cuda_lib
    sizes, N, K = [37, 91, 50], 130, 200
    off = offsets_of(sizes)
    rng = np.random.default_rng(3)
    A = torch.from_numpy(rng.standard_normal((178, K))).to(torch.bfloat16).cuda()
    B = torch.from_numpy(rng.standard_normal((3, N, K))).to(torch.bfloat16).cuda()
    B2 = B.clone()
    A2 = A.clone()
    A2[37:128] = float("nan")
    A2[60] = float("inf")
    B2[1] = float("inf")
    outs = []
    for a, b in ((A, B), (A2, B2)):
        C = torch.empty(178, N, dtype=torch.bfloat16, device="cuda")
        g.gemm_grouped(3, 178, N, K, BF16, torch.from_numpy(off).int().cuda(), a, K, 1, b, N * K, 1, K, C, N, BF16,
                       1.0, 0.0, None, 0)
        outs.append(C)
    assert torch.equal(outs[0][:37], outs[1][:37]) and torch.equal(outs[0][128:], outs[1][128:])
    assert not torch.isfinite(outs[1][37:128]).any()


def test_own_stream_and_repeat(cuda_lib):
    """On a side stream, behind work that fills its inputs there; twice, the same bits."""
    g = cuda_lib
    s = torch.cuda.Stream()
    a = run_grouped(g, SPLITS["tiles"], 256, 512, BF16, F32, seed=9, stream=s)
    b = run_grouped(g, SPLITS["tiles"], 256, 512, BF16, F32, seed=9)
    np.testing.assert_array_equal(a[0], b[0])


def test_offsets_out_of_range_are_clamped(cuda_lib):
    """Wild offsets touch nothing outside the arrays."""
    g = cuda_lib
    M, N, K = 100, 64, 64
    A = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    B = torch.ones(3, N, K, dtype=torch.bfloat16, device="cuda")
    C = torch.full((M + 64, N), CANARY, device="cuda")
    off = torch.tensor([-5, 40, 1 << 30, 7], dtype=torch.int32, device="cuda")
    g.gemm_grouped(3, M, N, K, BF16, off, A, K, 1, B, N * K, 1, K, C, N, F32, 1.0, 0.0, None, 0)
    assert g.gemm_device_status() == 0
    assert bool((C[:M] == K).all()) and bool((C[M:] == CANARY).all())
    W = torch.full((3 * N * K + 64,), CANARY, device="cuda")
    g.gemm_grouped_wgrad(3, M, N, K, BF16, off, A, K, 1, A, K, 1, W, N * K, K, F32, 1.0, 0.0)
    assert g.gemm_device_status() == 0
    assert bool((W[3 * N * K:] == CANARY).all())
    assert W[0] == 40 and W[N * K] == 60 and W[2 * N * K] == 0


# ------------------------------------------------------------ weight gradient --

def run_wgrad(g, sizes, M, N, ab, out, *, seed=0, integer=False, alpha=1.0, beta=0.0, pad=0, first=0, after=0,
              a_sum=True, gap=5, row_fast=False, poison=False):
    rng = np.random.default_rng(seed)
    G, off = len(sizes), offsets_of(sizes, first)
    T = int(off[-1]) + after

    def operand(cols):
        v = values(rng, (T, cols), integer)
        if poison:  # rows of no group
            v[:first] = np.nan
            v[int(off[-1]):] = np.inf
        if row_fast:
            t, back = to_dev(v.T, ab, (T + 7) // 8 * 8 + 1)
            return t, back.T, 1, (T + 7) // 8 * 8 + 1
        ld = (cols + 7) // 8 * 8 + pad
        t, back = to_dev(v, ab, ld)
        return t, back, ld, 1

    A, Av, sar, sam = operand(M)
    D, Dv, sdr, sdn = operand(N)
    ldc = N + 3
    scg = M * ldc + gap
    C = torch.full((G * scg + 16,), CANARY, dtype=DT[out])
    C0 = torch.from_numpy(values(rng, (G, M, N), integer)).to(DT[out])
    view = C[:G * scg].view(G, scg)[:, :M * ldc].view(G, M, ldc)
    view[:, :, :N] = C0 if beta != 0.0 else torch.full_like(C0, float("nan"))
    before = C.clone()
    s0 = torch.from_numpy(values(rng, (G, M), integer)).float() if a_sum else None
    s = s0.clone().cuda() if a_sum else None
    if a_sum and beta == 0.0:
        s.fill_(float("nan"))
    C = C.cuda()
    g.gemm_grouped_wgrad(G, T, M, N, ab, torch.from_numpy(off).int().cuda(), A, sar, sam, D, sdr, sdn, C, scg, ldc,
                         out, alpha, beta, a_sum=s)
    path = g.gemm_last_launch()["path"]
    assert g.gemm_device_status() == 0
    C = C.cpu()
    got = C[:G * scg].view(G, scg)[:, :M * ldc].view(G, M, ldc)
    bgot = before[:G * scg].view(G, scg)
    assert torch.equal(got[:, :, N:], bgot[:, :M * ldc].view(G, M, ldc)[:, :, N:])
    assert torch.equal(C[:G * scg].view(G, scg)[:, M * ldc:], bgot[:, M * ldc:]) and bool((C[G * scg:] == CANARY).all())
    Y, DD, S, SD = og.wgrad_reference(off, Av, Dv, alpha, beta, C0.double().numpy(),
                                      s0.double().numpy() if a_sum else None)
    return (got[:, :, :N].double().numpy(), Y, DD, path,
            (s.cpu().double().numpy(), S, SD) if a_sum else None)


@pytest.mark.parametrize("split", SPLITS, ids=str)
@pytest.mark.parametrize("M,N", [(1, 1), (72, 40), (300, 264), (129, 500)], ids=str)
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_wgrad_integer_exact(cuda_lib, split, M, N, ab):
    """Ragged sums over rows, empty groups zero, neighbouring rows' NaN and infinities never read into a sum."""
    got, want, _, path, sums = run_wgrad(cuda_lib, SPLITS[split], M, N, ab, F32, integer=True, seed=M + N, pad=8,
                                         first=3, after=9, poison=True)
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(sums[0], sums[1])


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("beta", [0.0, 1.0, 0.5])
def test_wgrad_accumulates(cuda_lib, out, beta):
    got, want, D, _, sums = run_wgrad(cuda_lib, SPLITS["ragged"], 136, 264, BF16, out, alpha=0.5, beta=beta, seed=2)
    check(got, want, D, out, 1.0)
    check(sums[0], sums[1], sums[2], F32, 1.0)


def test_wgrad_not_finite_stays_in_its_group(cuda_lib):
    """A group of NaN between two others, sharing k-blocks with neither's sum."""
    g = cuda_lib
    sizes, M, N = [37, 91, 50], 136, 72
    off = torch.from_numpy(offsets_of(sizes)).int().cuda()
    rng = np.random.default_rng(4)
    A = torch.from_numpy(rng.standard_normal((178, M))).half().cuda()
    D = torch.from_numpy(rng.standard_normal((178, N))).half().cuda()
    A2, D2 = A.clone(), D.clone()
    A2[37:128] = float("nan")
    D2[37:128] = float("inf")
    outs = []
    for a, d in ((A, D), (A2, D2)):
        C = torch.empty(3, M, N, device="cuda")
        g.gemm_grouped_wgrad(3, 178, M, N, F16, off, a, M, 1, d, N, 1, C, M * N, N, F32, 1.0, 0.0)
        outs.append(C)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][2], outs[1][2])
    assert torch.isnan(outs[1][1]).all()


@pytest.mark.parametrize("kw", [dict(row_fast=True), dict(pad=3)], ids=str)
def test_wgrad_strides_tma_cannot_read(cuda_lib, kw):
    got, want, _, path, _ = run_wgrad(cuda_lib, SPLITS["ragged"], 70, 90, BF16, F32, integer=True, **kw)
    np.testing.assert_array_equal(got, want)
    assert path == cuda_lib.PATH_SIMT


def test_wgrad_fp32_and_no_product(cuda_lib):
    got, want, D, path, sums = run_wgrad(cuda_lib, SPLITS["ragged"], 70, 90, F32, F32)
    check(got, want, D, F32, 1.0)
    assert path == cuda_lib.PATH_SIMT
    got, want, D, path, sums = run_wgrad(cuda_lib, SPLITS["ragged"], 70, 90, F16, F32, alpha=0.0, beta=3.0)
    check(got, want, D, F32, 1.0)
    check(sums[0], sums[1], sums[2], F32, 1.0)
    assert path == cuda_lib.PATH_EPILOGUE_ONLY


def test_gradients_by_differences(cuda_lib):
    """The three gradients of L = sum(P * (x W^T + b)) by central differences of the forward product.

    L is linear in each argument, so a difference has no truncation error; with every output and partial sum a
    multiple of 2^-6 below 2^18, fp32 holds it exactly and the differences equal the gradients exactly."""
    g = cuda_lib
    rng = np.random.default_rng(8)
    sizes, N, K = [9, 0, 40, 15], 48, 72
    G, M = len(sizes), sum(sizes)
    off = torch.from_numpy(offsets_of(sizes)).int().cuda()
    x = torch.from_numpy(rng.integers(-3, 4, (M, K))).to(torch.bfloat16).cuda()
    w = torch.from_numpy(rng.integers(-3, 4, (G, N, K))).to(torch.bfloat16).cuda()
    b = torch.from_numpy(rng.integers(-3, 4, (G, N))).float().cuda()
    p = torch.from_numpy(rng.integers(-3, 4, (M, N))).to(torch.bfloat16).cuda()

    def loss(x, w, b):
        y = torch.empty(M, N, device="cuda")
        g.gemm_grouped(G, M, N, K, BF16, off, x, K, 1, w, N * K, 1, K, y, N, F32, 1.0, 0.0, b, g.EPI_BIAS)
        return (y.double() * p.double()).sum().item()

    dx = torch.empty(M, K, device="cuda")
    g.gemm_grouped(G, M, K, N, BF16, off, p, N, 1, w, N * K, K, 1, dx, K, F32, 1.0, 0.0, None, 0)
    dw = torch.empty(G, N, K, device="cuda")
    db = torch.empty(G, N, device="cuda")
    g.gemm_grouped_wgrad(G, M, N, K, BF16, off, p, N, 1, x, K, 1, dw, N * K, K, F32, 1.0, 0.0, a_sum=db)
    h = 0.5
    for t, grad in ((0, dx), (1, dw), (2, db)):
        for _ in range(12):
            idx = tuple(int(rng.integers(0, n)) for n in grad.shape)
            args = [x.clone(), w.clone(), b.clone()], [x.clone(), w.clone(), b.clone()]
            args[0][t][idx] += h
            args[1][t][idx] -= h
            assert (loss(*args[0]) - loss(*args[1])) / (2 * h) == grad[idx].item()


def test_offsets_past_32_bits(cuda_lib):
    """A weight block and an output block whose element offsets pass 2^31."""
    g = cuda_lib
    G, N, K = 2, 72, 64
    far = (1 << 31) + 4096
    B = torch.zeros(far + N * K, dtype=torch.float16, device="cuda")
    A = torch.ones(20, K, dtype=torch.float16, device="cuda")
    B[:N * K] = 1
    B[far:] = 2
    off = torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda")
    C = torch.empty(20, N, device="cuda")
    g.gemm_grouped(G, 20, N, K, F16, off, A, K, 1, B, far, 1, K, C, N, F32, 1.0, 0.0, None, 0)
    assert bool((C[:7] == K).all()) and bool((C[7:] == 2 * K).all())
    g.gemm_grouped_wgrad(G, 20, K, K, F16, off, A, K, 1, A, K, 1, B, far, K, F16, 1.0, 0.0)
    assert g.gemm_device_status() == 0
    assert bool((B[:K * K] == 7).all()) and bool((B[far:far + K * K] == 13).all())
