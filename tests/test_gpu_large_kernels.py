"""The grouped and 8-bit kernels for large calls, each named by the launch record: every epilogue and output type on the
SM-pair kernels, large group tables, long groups of the weight gradient over more tiles than SM pairs, the widths of the
8-bit kernel, the largest sums, streams.  Bounds as in test_gpu_grouped.py; integer sums exact."""
import numpy as np
import pytest
import torch

from test_gpu_grouped import (BF16, CANARY, DT, F16, F32, NAMES, SPLITS, check, offsets_of, run_grouped, run_wgrad)
from test_gpu_i8 import run_i8

pytestmark = pytest.mark.gpu

PAIR, FEW = 2, 3  # gemm_launch_info_t kinds


def kind(g):
    return g.gemm_last_launch()["kind"]


# ------------------------------------------------------------- which kernel --

@pytest.mark.parametrize("rows,tile", [(1, 8), (5, 8), (8, 8), (9, 16), (16, 16), (17, 32), (32, 32)])
def test_few_rows_by_name(cuda_lib, rows, tile):
    g = cuda_lib
    got, want, _, path = run_grouped(g, [rows], 300, 520, BF16, F32, integer=True, seed=rows)
    info = g.gemm_last_launch()
    assert (path, info["kind"], info["bn"]) == (g.PATH_SIMT, FEW, tile)
    np.testing.assert_array_equal(got, want)
    got, want, _, path = run_i8(g, [rows], 300, 1040, F32, kind="positive", grouped=False, seed=rows)
    info = g.gemm_last_launch()
    assert (path, info["kind"], info["bn"]) == (g.PATH_SIMT, FEW, tile)
    np.testing.assert_array_equal(got, want.astype(np.float32))


def test_cuda_cores_by_name(cuda_lib):
    g = cuda_lib
    run_grouped(g, [5], 300, 520, BF16, F32, integer=True, b_shift=1)
    assert g.gemm_last_launch()["path"] == g.PATH_SIMT and kind(g) == 0
    run_i8(g, [5], 300, 520, F32, align=1, grouped=False)
    assert g.gemm_last_launch()["path"] == g.PATH_SIMT and kind(g) == 0


# -------------------------------------------------------- grouped, SM pairs --

@pytest.mark.parametrize("trans", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("epi", range(6))
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_pair_epilogues(cuda_lib, epi, out, ab, trans):
    """alpha, beta * C, bias, activation and row scale; K in one accumulator and in three."""
    for K in (328, 1160):
        got, want, D, _ = run_grouped(cuda_lib, SPLITS["ragged"], 1513, K, ab, out, epi=epi, alpha=0.75, beta=0.5,
                                      row_scale=True, seed=epi + K, trans=trans, first=2, after=4)
        assert kind(cuda_lib) == PAIR
        check(got, want, D, out)


@pytest.mark.parametrize("ldc_pad", [0, 1, 2, 5])
@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
def test_pair_output_pitch(cuda_lib, ldc_pad, out):
    for N in (2000, 2003):
        got, want, D, _ = run_grouped(cuda_lib, [70, 0, 41, 300], N, 72, F16, out, ldc_pad=ldc_pad, epi=4, seed=N)
        assert kind(cuda_lib) == PAIR
        check(got, want, D, out)


def test_pair_not_finite_stays_in_its_rows(cuda_lib):
    """Tiles of 32 columns whose loads reach the next group's rows."""
    g = cuda_lib
    sizes, N, K = [37, 91, 50], 2600, 200
    off = torch.from_numpy(offsets_of(sizes)).int().cuda()
    rng = np.random.default_rng(3)
    A = torch.from_numpy(rng.standard_normal((178, K))).to(torch.bfloat16).cuda()
    B = torch.from_numpy(rng.standard_normal((3, N, K))).to(torch.bfloat16).cuda()
    A2, B2 = A.clone(), B.clone()
    A2[37:128] = float("nan")
    A2[60] = float("inf")
    B2[1] = float("inf")
    outs = []
    for a, b in ((A, B), (A2, B2)):
        C = torch.empty(178, N, dtype=torch.bfloat16, device="cuda")
        g.gemm_grouped(3, 178, N, K, BF16, off, a, K, 1, b, N * K, 1, K, C, N, BF16, 1.0, 0.0, None, 0)
        assert kind(g) == PAIR
        outs.append(C)
    assert torch.equal(outs[0][:37], outs[1][:37]) and torch.equal(outs[0][128:], outs[1][128:])
    assert not torch.isfinite(outs[1][37:128]).any()


def many_groups(G, rows, seed):
    """G sizes that sum to `rows`, empty ones among them."""
    cuts = np.sort(np.random.default_rng(seed).integers(0, rows + 1, size=G - 1))
    return np.diff(np.concatenate([[0], cuts, [rows]])).tolist()


@pytest.mark.parametrize("G", [143, 144, 200, 1024])
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_many_groups(cuda_lib, G, ab):
    """Group tables beside which the ring has six stages, up to the largest; deep enough to go round it twice."""
    sizes = many_groups(G, 3 * G, G)
    got, want, _, _ = run_grouped(cuda_lib, sizes, 48, 1000, ab, F32, integer=True, trans=True, seed=G, first=1)
    assert kind(cuda_lib) == PAIR
    np.testing.assert_array_equal(got, want)
    got, want, _, _ = run_grouped(cuda_lib, sizes, 48, 200, ab, F32, integer=True, seed=G)
    np.testing.assert_array_equal(got, want)
    got, want, _, _, sums = run_wgrad(cuda_lib, sizes, 24, 40, ab, F32, integer=True, seed=G, first=2, after=70,
                                      poison=True)
    assert kind(cuda_lib) == PAIR
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(sums[0], sums[1])


# ---------------------------------------------------------- weight gradient --

@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("ab", [F16, BF16], ids=NAMES.get)
def test_wgrad_long_groups(cuda_lib, ab, out):
    """100 tiles; groups of 10 to 32 k-blocks, none a multiple of 64 rows, so accumulators, ring and the cleared
    blocks' barriers come round several times."""
    sizes = [1999, 0, 601, 1300, 777]
    got, want, _, _, sums = run_wgrad(cuda_lib, sizes, 1100, 1000, ab, out, integer=True, seed=out, first=5, after=33,
                                      poison=True)
    assert kind(cuda_lib) == PAIR
    want = torch.from_numpy(want).to(DT[out]).double().numpy()  # integers: exact sums, one rounding
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(sums[0], sums[1])


@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
def test_wgrad_accumulates_long_groups(cuda_lib, out):
    got, want, D, _, sums = run_wgrad(cuda_lib, [1999, 0, 601, 1300, 777], 300, 520, BF16, out, alpha=0.5, beta=1.0,
                                      seed=7, after=3)
    assert kind(cuda_lib) == PAIR
    check(got, want, D, out, 1.0)
    check(sums[0], sums[1], sums[2], F32, 1.0)


# ------------------------------------------------------------ 8-bit, SM pairs --

@pytest.mark.parametrize("out", [F32, F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("epi", range(6))
@pytest.mark.parametrize("sizes", [[330], [0, 133, 1, 90, 200]], ids=["dense", "grouped"])
def test_i8_pair_epilogues(cuda_lib, out, epi, sizes):
    """K in one accumulator (exact in fp32) and in three (integers in registers)."""
    for K in (333, 2500):
        got, want, D, path = run_i8(cuda_lib, sizes, 2603, K, out, epi=epi, alpha=0.25, beta=0.5, scales="random",
                                    grouped=len(sizes) > 1, seed=K + epi)
        assert path == cuda_lib.PATH_TCGEN05
        check(got, want, D, out)


@pytest.mark.parametrize("ldc_pad", [0, 1, 2])
@pytest.mark.parametrize("out", [F16, BF16], ids=NAMES.get)
def test_i8_pair_output_pitch(cuda_lib, ldc_pad, out):
    for N in (2560, 2563):
        got, want, D, path = run_i8(cuda_lib, [300], N, 64, out, ldc_pad=ldc_pad, scales="random", grouped=False)
        assert path == cuda_lib.PATH_TCGEN05
        check(got, want, D, out)


def i8_on_gpu(g, sizes, N, K, seed):
    """One fp32 call without scales on random codes, its launch record, and the exact sums (float64 on the GPU)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    G, off = len(sizes), offsets_of(sizes)
    M, ld = int(off[-1]), (K + 15) // 16 * 16
    X = torch.randint(-128, 128, (M, ld), dtype=torch.int8, device="cuda", generator=gen)
    W = torch.randint(-128, 128, (G, N, ld), dtype=torch.int8, device="cuda", generator=gen)
    C = torch.full((M, N), CANARY, device="cuda")
    g.gemm_i8_grouped(G, M, N, K, torch.from_numpy(off).int().cuda(), X, ld, None, W, N * ld, ld, None, C, N, F32, 1.0,
                      0.0, None, 0)
    info = g.gemm_last_launch()
    assert g.gemm_device_status() == 0
    want = torch.cat([X[off[e]:off[e + 1], :K].double() @ W[e, :, :K].double().T for e in range(G)])
    return C, want.float(), info


@pytest.mark.parametrize("sizes,N,K,most", [([200], 2600, 1300, 64), ([600], 2304, 1300, 128), ([8192], 2304, 700, 192),
                                            ([500, 0, 700, 3, 129], 2600, 1100, None)], ids=str)
def test_i8_widths(cuda_lib, sizes, N, K, most):
    C, want, info = i8_on_gpu(cuda_lib, sizes, N, K, 1)
    assert info["path"] == cuda_lib.PATH_TCGEN05 and most in (None, info["bn"]), info
    assert torch.equal(C, want)


@pytest.mark.parametrize("G", [143, 200, 1024])
@pytest.mark.parametrize("per", [6, 100, 190])
def test_i8_many_groups(cuda_lib, G, per):
    """Tiles of 32 to 192 rows beside large group tables: fewer stages or slots, each used many times."""
    sizes = many_groups(G, per * G, G) if per == 6 else np.random.default_rng(G).integers(per - 20, per + 3, G).tolist()
    C, want, info = i8_on_gpu(cuda_lib, sizes, 260, 1300, G)
    assert info["path"] == cuda_lib.PATH_TCGEN05
    assert torch.equal(C, want)


@pytest.mark.parametrize("M", [200, 600])
def test_i8_pair_largest_sums(cuda_lib, M):
    """K at its limit, every code -128, on the pair kernel: 128 accumulators of 2^24 each, added as integers."""
    g = cuda_lib
    N, K = 2304, g.I8_MAX_K
    X = torch.full((M, K + 1), -128, dtype=torch.int8, device="cuda")
    W = torch.full((N, K + 1), -128, dtype=torch.int8, device="cuda")
    C = torch.empty(M, N, device="cuda")
    g.gemm_i8(M, N, K, X, K + 1, None, W, K + 1, None, C, N, F32, 1.0, 0.0, None, 0)
    assert g.gemm_last_launch()["path"] == g.PATH_TCGEN05 and g.gemm_device_status() == 0
    assert bool((C == float(np.float32(16384 * K))).all())


# ------------------------------------------------------------------- streams --

def test_inputs_filled_on_the_same_stream(cuda_lib):
    """Every entry point behind work of its stream that has not run when the call returns: a wait of many
    milliseconds, then the copies that make the inputs (NaN and -1 until then)."""
    g = cuda_lib
    G, M, N, K = 3, 600, 1600, 512
    off = torch.tensor([0, 100, 350, 600], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    w = torch.randn(G, N, K, device="cuda", generator=gen).bfloat16()
    dy = torch.randn(M, N, device="cuda", generator=gen).bfloat16()
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=gen)
    qw = torch.randint(-127, 128, (G, N, K), dtype=torch.int8, device="cuda", generator=gen)

    def late(stream, check=True):
        """Results of the five calls, their inputs filled on `stream` behind a wait."""
        xi, wi, di, qi, qwi, oi = (torch.full_like(t, -1 if t.dtype == torch.int8 else 0 if t.dtype == torch.int32
                                                   else float("nan")) for t in (x, w, dy, q, qw, off))
        y, dw = torch.empty(M, N, device="cuda"), torch.empty(G, N, K, device="cuda")
        db, yi = torch.empty(G, N, device="cuda"), torch.empty(M, N, device="cuda")
        few = torch.empty(4, N, device="cuda")
        codes, scale = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        torch.cuda.synchronize()
        done = torch.cuda.Event()
        with torch.cuda.stream(stream):
            torch.cuda._sleep(60_000_000)
            for a, b in ((xi, x), (wi, w), (di, dy), (qi, q), (qwi, qw), (oi, off)):
                a.copy_(b)
            g.gemm_grouped(G, M, N, K, BF16, oi, xi, K, 1, wi, N * K, 1, K, y, N, F32, 1.0, 0.0, None, 0)
            g.gemm_grouped_wgrad(G, M, N, K, BF16, oi, di, N, 1, xi, K, 1, dw, N * K, K, F32, 1.0, 0.0, a_sum=db)
            g.gemm_i8_grouped(G, M, N, K, oi, qi, K, None, qwi, N * K, K, None, yi, N, F32, 1.0, 0.0, None, 0)
            g.gemm_i8(4, N, K, qi, K, None, qwi, K, None, few, N, F32, 1.0, 0.0, None, 0)
            g.gemm_i8_quantize(M, K, BF16, xi, K, codes, K, scale)
            done.record()
            assert not (check and done.query()), "the calls waited for the stream"
        stream.synchronize()
        assert g.gemm_device_status(stream) == 0
        return y, dw, db, yi, few, codes, scale

    late(torch.cuda.Stream(), False)  # loads the kernels
    a, b = late(torch.cuda.Stream()), late(torch.cuda.default_stream())
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    want = torch.cat([x[r].double() @ w[e].double().T for e, r in enumerate((slice(0, 100), slice(100, 350),
                                                                           slice(350, 600)))])
    assert bool(((a[0].double() - want).abs() <= 1e-5 * 40 * K).all())  # |x w| <= 5 * 5 a term, well below 40 K
    assert torch.equal(a[3].double(), torch.cat([q[r].double() @ qw[e].double().T for e, r in enumerate(
        (slice(0, 100), slice(100, 350), slice(350, 600)))]))
