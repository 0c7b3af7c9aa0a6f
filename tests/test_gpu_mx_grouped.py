"""GPU tests of the block-scaled product grouped by expert (gemm_mx_grouped) against float64.

Codes whose values are small integers, with scales per row and block that are powers of two of a narrow range, have
exact fp32 sums: outputs bit for bit.  Others are held to |got - want| <= u |want| + n 2^-23 D s: u the output's
roundoff, n the matrix instructions along K (32 or 64 deep) plus one, each of which the tensor cores round by
cutting off to within a unit in the last place of a sum that D bounds, s the activation's largest slope.
"""
import numpy as np
import pytest
import torch

import oracle.mx_rows as om
from oracle import grouped as og

pytestmark = pytest.mark.gpu

F32, F16, BF16 = 0, 1, 2
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
ROUNDOFF = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
E4M3, E2M1 = 0, 1
PER = {E4M3: 1, E2M1: 2}
CANARY = 77.0

SPLITS = {"one": [5], "ragged": [0, 1, 33, 0, 130, 7, 0], "tiles": [224, 225, 255, 64, 96], "wide": [700, 449],
          "many": [3] * 40 + [0] * 20 + [1] * 17, "empty": [0, 0, 0], "row": [1]}


def coded(rng, shape, K, elem, kind):
    """Codes (one per element), scales and values of shape[0] x ... rows of K."""
    n = int(np.prod(shape))
    if kind == "integer":
        vals = np.array([-2, -1, -0.0, 0, 1, 2]) if elem == E2M1 else np.arange(-4.0, 5.0)
        pick = rng.integers(0, len(vals), (n, K), dtype=np.uint8)
        scale = rng.integers(127, 130, (n, K // 32))
        return om.nearest_codes(vals, elem)[pick], scale, vals[pick] * np.repeat(2.0 ** (scale - 127), 32, 1)
    codes, scale = om.quantize_reference(rng.standard_normal((n, K)) * 10.0 ** rng.uniform(-2, 2, (n, 1)), elem)
    return codes, scale, om.values_of(codes, scale, elem)


def pitched(a, pitch, fill):
    out = np.full((a.shape[0], pitch), fill, np.uint8)
    out[:, :a.shape[1]] = a
    return torch.from_numpy(out).cuda()


def run(g, sizes, N, K, elem, out, *, kind="integer", seed=0, epi=0, alpha=1.0, beta=0.0, row_scale=False, pad=0, first=0,
        after=0, ldc_pad=3, nan_rows=False, offsets=True, stream=None):
    rng = np.random.default_rng(seed)
    G, off = len(sizes), np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int64)
    M = int(off[-1]) + after
    xc, xs, xv = coded(rng, (M,), K, elem, kind)
    wc, ws, wv = coded(rng, (G, N), K, elem, kind)
    if nan_rows:  # rows of no group: NaN scales and, in E4M3, NaN elements
        xs[:first], xs[int(off[-1]):] = 255, 255
        if elem == E4M3:
            xc[int(off[-1]):] = 127
    qp, sp = (K // PER[elem] + 15) // 16 * 16 + 16 * pad, (K // 32 + 15) // 16 * 16 + 16 * pad
    X, W = pitched(om.packed(xc, elem), qp, 0xFF), pitched(om.packed(wc, elem), qp, 0xFF)
    XS, WS = pitched(xs, sp, 0xFF), pitched(ws, sp, 0xFF)
    ldc = N + ldc_pad
    C0 = torch.from_numpy(rng.integers(-4, 5, (M, N)).astype(np.float64)).to(DT[out])
    C = torch.full((M + 2, ldc), CANARY, dtype=DT[out])
    C[1 + first:1 + int(off[-1]), :N] = C0[first:int(off[-1])] if beta else float("nan")
    before = C.clone()
    C = C.cuda()
    bias = torch.from_numpy(rng.integers(-4, 5, (G, N)).astype(np.float64)).float() if epi else None
    rs = torch.from_numpy(rng.choice([0.5, 1.0, 2.0], size=M)).float() if row_scale else None
    g.gemm_mx_grouped(G, M, N, K, elem, torch.from_numpy(off).int().cuda() if offsets else None, X, qp * PER[elem], XS, sp, W,
                      N * qp * PER[elem], qp * PER[elem], WS, N * sp, sp, C.data_ptr() + ldc * C.element_size(), ldc, out,
                      alpha, beta, None if bias is None else bias.cuda(), epi, None if rs is None else rs.cuda(), stream)
    assert g.gemm_device_status(stream) == 0
    C = C.cpu()
    keep = np.ones(C.shape, dtype=bool)
    keep[1 + first:1 + int(off[-1]), :N] = False
    assert torch.equal(C[torch.from_numpy(keep)], before[torch.from_numpy(keep)]), "wrote outside its rows"
    Y, D = og.grouped_reference(off, xv, wv.reshape(G, N, K).transpose(0, 2, 1), epi, alpha, beta,
                                C0.double().numpy() if beta else None, None if bias is None else bias.double().numpy(),
                                None if rs is None else rs.double().numpy())
    sl = slice(first, int(off[-1]))
    return C[1:M + 1, :N].double().numpy()[sl], Y[sl], D[sl]


def check(got, want, D, out, K, elem, slope=1.13):
    n = -(-K // (32 * PER[elem])) + 1
    bound = ROUNDOFF[out] * np.abs(want) + n * 2.0 ** -23 * slope * D + (2.0 ** -25 if out == F16 else 0.0) + 5e-7 * slope * D
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst by {np.nanmax(np.abs(got - want) - bound):.3e}"


@pytest.mark.parametrize("split", SPLITS, ids=str)
@pytest.mark.parametrize("N,K", [(1, 32), (72, 64), (300, 512), (257, 1056), (600, 2080)], ids=str)
@pytest.mark.parametrize("elem", [E2M1, E4M3], ids=["e2m1", "e4m3"])
def test_integer_exact(cuda_lib, split, N, K, elem):
    """A wrong row, channel, group, scale, byte or k tail shows as a wrong integer."""
    got, want, _ = run(cuda_lib, SPLITS[split], N, K, elem, F32, seed=N + K, pad=K % 64 // 32, first=3, after=5,
                       nan_rows=True)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("elem", [E2M1, E4M3], ids=["e2m1", "e4m3"])
@pytest.mark.parametrize("rows", list(range(1, 34)) + [63, 64, 65, 95, 97, 127, 128, 129, 160, 191, 192, 193, 223, 224])
def test_every_width(cuda_lib, elem, rows):
    got, want, _ = run(cuda_lib, [rows], 256, 512, elem, F32, seed=rows, after=40, nan_rows=True)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("split,N,K", [("ragged", 300, 512), ("wide", 513, 4096), ("many", 1024, 1056)])
@pytest.mark.parametrize("elem", [E2M1, E4M3], ids=["e2m1", "e4m3"])
@pytest.mark.parametrize("out", [F32, F16, BF16])
def test_quantised_values(cuda_lib, split, N, K, elem, out):
    got, want, D = run(cuda_lib, SPLITS[split], N, K, elem, out, kind="normal", seed=K)
    if out == F16:  # values past its largest are infinities
        big = np.abs(want) >= 65504
        got, want, D = got[~big], want[~big], D[~big]
    check(got, want, D, out, K, elem)


@pytest.mark.parametrize("epi", range(6))
@pytest.mark.parametrize("out", [F32, BF16])
def test_epilogues(cuda_lib, epi, out):
    got, want, D = run(cuda_lib, SPLITS["ragged"], 136, 256, E2M1, out, kind="normal", epi=epi, alpha=0.5, beta=0.25,
                       row_scale=True, seed=epi)
    check(got, want, D, out, 256, E2M1)


@pytest.mark.parametrize("alpha,beta,K", [(0.0, 0.5, 256), (0.0, 0.0, 256), (1.0, 0.5, 0), (1.0, 0.0, 0)])
def test_without_a_product(cuda_lib, alpha, beta, K):
    """alpha == 0 and K == 0: bias, beta C and the activation alone; operands may be anything."""
    g = cuda_lib
    off = torch.tensor([0, 5, 5, 300], dtype=torch.int32, device="cuda")
    C = torch.arange(300 * 40, device="cuda").view(300, 40).remainder(13).float()
    c0 = C.clone()
    bias = torch.randn(3, 40, device="cuda")
    g.gemm_mx_grouped(3, 300, 40, K, E2M1, off, None, 0, None, 0, None, 0, 0, None, 0, 0, C, 40, F32, alpha, beta, bias,
                      g.EPI_BIAS_RELU)
    assert g.gemm_device_status() == 0
    e = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor([5, 0, 295], device="cuda"))
    assert torch.equal(C, torch.relu(beta * c0 + bias[e]))


@pytest.mark.parametrize("elem", [E2M1, E4M3], ids=["e2m1", "e4m3"])
def test_dense_call_and_the_dense_kernel(cuda_lib, elem):
    """One group without offsets is gemm_mx's product: the same integers."""
    g = cuda_lib
    got, want, _ = run(g, [333], 520, 512, elem, F32, seed=4, offsets=False)
    np.testing.assert_array_equal(got, want)


def test_nan_scales_show_in_their_rows_and_columns_alone(cuda_lib):
    g = cuda_lib
    M, N, K = 300, 300, 1024
    x, w = (torch.full((r, K // 2), 0x22, dtype=torch.uint8, device="cuda") for r in (M, N))
    xs, ws = (torch.full((r, K // 32), 127, dtype=torch.uint8, device="cuda") for r in (M, N))
    xs[17, 3], xs[250, 31], ws[40, 0], ws[299, 20] = 255, 255, 255, 255
    C = torch.empty(M, N, device="cuda")
    g.gemm_mx_grouped(1, M, N, K, E2M1, None, x, K, xs, 32, w, 0, K, ws, 0, 32, C, N, F32, 1.0, 0.0, None, 0)
    want = torch.full((M, N), float(K), device="cuda")
    want[[17, 250]] = float("nan")
    want[:, [40, 299]] = float("nan")
    assert torch.equal(torch.isnan(C), torch.isnan(want)) and (C[~torch.isnan(C)] == K).all()


def test_offsets_that_fall_or_leave_the_arrays(cuda_lib):
    """Clamped and raised as in gemm_grouped: no row outside 0 .. M-1, none twice, no group's guard touched."""
    g = cuda_lib
    M, N, K = 100, 64, 64
    x, w = (torch.full((r, K // 2), 0x22, dtype=torch.uint8, device="cuda") for r in (M, 4 * N))
    xs, ws = (torch.full((r, 16), 127, dtype=torch.uint8, device="cuda") for r in (M, 4 * N))
    for off in ([-5, 30, 20, 500, 2 ** 31 - 1], [90, 10, 50, 20, 60], [200, 300, 400, 500, 600]):
        C = torch.full((M + 2, N), CANARY, device="cuda")
        g.gemm_mx_grouped(4, M, N, K, E2M1, torch.tensor(off, dtype=torch.int32, device="cuda"), x, K, xs, 16, w, N * K, K,
                          ws, N * 16, 16, C[1:], N, F32, 1.0, 0.0, None, 0)
        assert g.gemm_device_status() == 0
        assert (C[0] == CANARY).all() and (C[M + 1] == CANARY).all()
        assert ((C == CANARY) | (C == K)).all()


@pytest.mark.parametrize("elem", [E2M1, E4M3], ids=["e2m1", "e4m3"])
def test_long_one_sided_sums(cuda_lib, elem):
    """8192 positive products: nothing cancels, and what the tensor cores cut off adds up to no more than the bound."""
    rng = np.random.default_rng(0)
    M, N, K, g = 48, 272, 8192, cuda_lib
    codes = [rng.integers(1, 8 if elem == E2M1 else 127, (r, K)) for r in (M, N)]
    scales = [rng.integers(120, 130, (r, K // 32)) for r in (M, N)]
    xv, wv = (om.values_of(c, s, elem) for c, s in zip(codes, scales))
    X, W = (torch.from_numpy(om.packed(c, elem)).cuda() for c in codes)
    XS, WS = (torch.from_numpy(s.astype(np.uint8)).cuda() for s in scales)
    C = torch.empty(M, N, device="cuda")
    g.gemm_mx_grouped(1, M, N, K, elem, None, X, K, XS, K // 32, W, 0, K, WS, 0, K // 32, C, N, F32, 1.0, 0.0, None, 0)
    want = xv @ wv.T
    check(C.cpu().double().numpy(), want, want, F32, K, elem)


def test_the_largest_table_and_single_rows(cuda_lib):
    """1024 groups; one row and one channel, whose pitches are not used and may be anything."""
    rng = np.random.default_rng(1)
    sizes = rng.integers(0, 4, 1024).tolist()
    got, want, _ = run(cuda_lib, sizes, 40, 64, E2M1, F32, seed=2)
    np.testing.assert_array_equal(got, want)
    g, K = cuda_lib, 96
    x, w = (torch.full((K // 2,), 0x22, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.full((K // 32,), 127, dtype=torch.uint8, device="cuda")
    C = torch.full((1,), float("nan"), device="cuda")
    g.gemm_mx_grouped(1, 1, 1, K, E2M1, None, x, K + 2, s, 3, w, 0, K + 6, s, 0, 5, C, 1, F32, 1.0, 0.0, None, 0)
    assert g.gemm_device_status() == 0 and C.item() == K


@pytest.mark.parametrize("elem", [E2M1, E4M3], ids=["e2m1", "e4m3"])
def test_the_same_call_gives_the_same_bits(cuda_lib, elem):
    """A row's result depends neither on the rows beside it nor on the run."""
    g, K, N, M = cuda_lib, 1024, 300, 900
    rng = np.random.default_rng(3)
    xc, xs, _ = coded(rng, (M,), K, elem, "normal")
    wc, ws, _ = coded(rng, (N,), K, elem, "normal")
    X, XS, W, WS = (torch.from_numpy(a).cuda() for a in (om.packed(xc, elem), xs.astype(np.uint8), om.packed(wc, elem),
                                                         ws.astype(np.uint8)))

    def product(rows):
        C = torch.empty(len(rows), N, device="cuda")
        g.gemm_mx_grouped(1, len(rows), N, K, elem, None, X[rows].contiguous(), K, XS[rows].contiguous(), K // 32, W, 0, K,
                          WS, 0, K // 32, C, N, F32, 1.0, 0.0, None, 0)
        return C

    whole = product(list(range(M)))
    assert torch.equal(whole, product(list(range(M))))
    for rows in ([5], [899, 3, 400], list(range(100, 350))):
        assert torch.equal(product(rows), whole[rows])


def test_row_blocks_past_2_to_the_31_elements(cuda_lib):
    """Outputs whose offsets pass 32 bits."""
    g, K, N, M = cuda_lib, 32, 2048, (1 << 20) + 5
    x = torch.full((M, 16), 0x22, dtype=torch.uint8, device="cuda")
    w = torch.full((N, 16), 0x22, dtype=torch.uint8, device="cuda")
    xs, ws = (torch.full((r, 16), 127, dtype=torch.uint8, device="cuda") for r in (M, N))
    xs[-1], ws[-1] = 128, 129
    C = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    g.gemm_mx_grouped(1, M, N, K, E2M1, None, x, K, xs, 16, w, 0, K, ws, 0, 16, C, N, BF16, 1.0, 0.0, None, 0)
    assert g.gemm_device_status() == 0
    assert (C[:-1, :-1] == K).all() and (C[-1, :-1] == 2 * K).all() and (C[:-1, -1] == 4 * K).all() and C[-1, -1] == 8 * K
