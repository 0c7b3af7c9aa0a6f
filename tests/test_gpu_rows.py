"""GPU tests of the movement of rows (gemm_rows_gather, gemm_rows_combine, gemm_rows_combine_grad) against float64.

A product's rounding is 2^-24 relative, a sum of n terms off by at most n 2^-24 of the terms' absolute sum, the
output's rounding by half a unit in the last place (fp16 also by 2^-25 among its subnormals).
"""
import numpy as np
import pytest
import torch

import oracle.route as orr

pytestmark = pytest.mark.gpu

F32, F16, BF16 = 0, 1, 2
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
HALF = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
U = 2.0 ** -24
CANARY = 77.0


def rows(rng, n, D, dtype, pad, shift=0):
    """n rows of normal values, pitch D + pad (NaN beyond D), `shift` elements into their allocation."""
    v = torch.from_numpy(rng.standard_normal((n, D))).to(DT[dtype])
    buf = torch.full((shift + n * (D + pad),), float("nan"), dtype=DT[dtype])
    buf[shift:].view(n, D + pad)[:, :D] = v
    return buf.cuda()[shift:].view(n, D + pad), v.double().numpy()


def blank(n, D, dtype, pad, fill=CANARY):
    return torch.full((n + 2, D + pad), fill, dtype=DT[dtype], device="cuda")


def inside(t, n, D):
    """Rows 1 .. n, columns below D; the rest must hold the canary."""
    t = t.cpu()
    assert (t[0] == CANARY).all() and (t[n + 1] == CANARY).all() and (t[:, D:] == CANARY).all()
    return t[1:n + 1, :D].double().numpy()


def order(rng, T, top, drop):
    """row (T x top, some -1) and source of the kept pairs in a random order."""
    keep = np.flatnonzero(rng.random(T * top) >= drop)
    perm = rng.permutation(keep)
    row, source = np.full(T * top, -1), np.full(T * top, -1)
    row[perm] = np.arange(perm.size)
    source[:perm.size] = perm
    return row.reshape(T, top), source, perm.size


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).int().cuda()


SHAPES = [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (5, 9, 264), (33, 4, 1001), (64, 6, 2056), (2, 17, 8200), (300, 3, 64)]


@pytest.mark.parametrize("T,top,D", SHAPES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_gather(cuda_lib, T, top, D, dtype, pad, shift):
    rng = np.random.default_rng(T + D)
    X, xv = rows(rng, T, D, dtype, pad, shift)
    row, source, n = order(rng, T, top, 0.3)
    R = T * top
    w = rng.standard_normal((T, top)).astype(np.float32)
    for weight in (None, w):
        Y = blank(R, D, dtype, pad)
        cuda_lib.gemm_rows_gather(R, D, T, top, dtype, X, D + pad, dev(source),
                                  None if weight is None else torch.from_numpy(weight).cuda(), Y[1:], D + pad)
        got = inside(Y, R, D)
        assert (got[n:] == CANARY).all(), "places without a pair were written"
        want = xv[source[:n] // top]
        if weight is None:
            np.testing.assert_array_equal(got[:n], want)
        else:
            want = want * w.reshape(-1)[source[:n], None].astype(np.float64)
            assert (np.abs(got[:n] - want) <= (U + HALF[dtype]) * np.abs(want) + 2.0 ** -25).all()


@pytest.mark.parametrize("T,top,D", SHAPES)
@pytest.mark.parametrize("y_dtype,out", [(F32, F32), (F32, F16), (F32, BF16), (F16, F32), (F16, F16), (BF16, F32),
                                         (BF16, BF16)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_combine(cuda_lib, T, top, D, y_dtype, out, pad, shift):
    """Tokens of which all pairs were dropped get beta times what they held; NaN rows that no pair names stay out."""
    rng = np.random.default_rng(T + D)
    R = T * top + 2
    Y, yv = rows(rng, R, D, y_dtype, pad, shift)
    row, _, n = order(rng, T, top, 0.4)
    row[T // 2] = -1
    if top > 1 and T > 1:
        row[0, 1] = R  # past the last row
    named = set(row.reshape(-1).tolist())
    for r in range(R):
        if r not in named:
            Y[r, :] = float("nan")
    w = rng.standard_normal((T, top)).astype(np.float32)
    for weight, beta in ((None, 0.0), (w, 0.0), (w, -0.5)):
        o = blank(T, D, out, pad)
        o0 = torch.from_numpy(rng.standard_normal((T, D))).to(DT[out])
        o[1:T + 1, :D] = o0.cuda() if beta else float("nan")
        cuda_lib.gemm_rows_combine(T, top, D, R, y_dtype, Y, D + pad, dev(row),
                                   None if weight is None else torch.from_numpy(weight).cuda(), beta, out, o[1:], D + pad)
        want, size = orr.combine_reference(yv, row, weight, beta, o0.double().numpy())
        got = inside(o, T, D)
        assert (np.abs(got - want) <= (top + 2) * U * size + HALF[out] * np.abs(want) + 2.0 ** -25).all()


@pytest.mark.parametrize("T,top,D", SHAPES)
@pytest.mark.parametrize("d_dtype,y_dtype", [(F32, F32), (F32, F16), (F32, BF16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_combine_gradient(cuda_lib, T, top, D, d_dtype, y_dtype, pad, shift):
    rng = np.random.default_rng(T + D)
    R = T * top + 3
    dO, ov = rows(rng, T, D, d_dtype, pad, shift)
    Y, yv = rows(rng, R, D, y_dtype, pad, shift)
    row, _, _ = order(rng, T, top, 0.3)
    row[T // 2] = -1
    w = rng.standard_normal((T, top)).astype(np.float32)
    named = row >= 0
    for weight in (None, w):
        wd = None if weight is None else torch.from_numpy(weight).cuda()
        dY, dw = blank(R, D, y_dtype, pad), torch.full((T * top + 4,), CANARY, device="cuda")
        args = (T, top, D, R, d_dtype, dO, D + pad, y_dtype)
        cuda_lib.gemm_rows_combine_grad(*args, Y, D + pad, dev(row), wd, dY[1:], D + pad, dw)
        got, gw = inside(dY, R, D), dw.cpu().double().numpy()
        assert (gw[T * top:] == CANARY).all()
        gw = gw[:T * top].reshape(T, top)
        wv = np.ones((T, top)) if weight is None else w.astype(np.float64)
        want = wv[named][:, None] * np.repeat(ov[:, None], top, 1)[named]
        assert (np.abs(got[row[named]] - want) <= (U + HALF[y_dtype]) * np.abs(want) + 2.0 ** -25).all()
        rest = np.setdiff1d(np.arange(R), row[named])
        assert (got[rest] == CANARY).all()
        terms = np.repeat(ov[:, None], top, 1)[named] * yv[row[named]]
        assert (np.abs(gw[named] - terms.sum(1)) <= (D + 1) * U * np.abs(terms).sum(1)).all()
        assert (gw[~named] == 0).all()
        # each alone gives the same bits; without dweight the rows are not read
        dY2, dw2 = blank(R, D, y_dtype, pad), torch.empty(T, top, device="cuda")
        cuda_lib.gemm_rows_combine_grad(*args, None, 0, dev(row), wd, dY2[1:], D + pad, None)
        cuda_lib.gemm_rows_combine_grad(*args, Y, D + pad, dev(row), wd, None, 0, dw2)
        assert torch.equal(dY, dY2) and torch.equal(dw[:T * top].view(T, top), dw2)


def test_gather_and_combine_are_each_others_gradients(cuda_lib):
    """<gather(x), y> = <x, combine(y)> exactly on small integers."""
    rng = np.random.default_rng(0)
    T, top, D = 50, 3, 136
    row, source, n = order(rng, T, top, 0.2)
    x, y = rng.integers(-3, 4, (T, D)), rng.integers(-3, 4, (T * top, D))
    X, Y = torch.from_numpy(x).float().cuda(), torch.from_numpy(y).float().cuda()
    G, C = torch.zeros_like(Y), torch.empty_like(X)
    cuda_lib.gemm_rows_gather(T * top, D, T, top, F32, X, D, dev(source), None, G, D)
    cuda_lib.gemm_rows_combine(T, top, D, T * top, F32, Y, D, dev(row), None, 0.0, F32, C, D)
    assert int((G.double() * Y.double()).sum()) == int((X.double() * C.double()).sum())


def test_rows_past_2_to_the_31_elements(cuda_lib):
    """Offsets in 64 bits: the last rows of an array of more than 2^31 elements."""
    D, R = 8192, 262144 + 3
    Y = torch.empty(R, D, dtype=torch.bfloat16, device="cuda")
    Y[-3:] = torch.arange(3 * D, device="cuda").view(3, D).remainder(100).bfloat16()
    row = torch.tensor([[R - 1, R - 2], [R - 3, -1]], dtype=torch.int32, device="cuda")
    out = torch.empty(2, D, dtype=torch.bfloat16, device="cuda")
    cuda_lib.gemm_rows_combine(2, 2, D, R, BF16, Y, D, row, None, 0.0, BF16, out, D)
    assert torch.equal(out[0], (Y[-1].float() + Y[-2].float()).bfloat16()) and torch.equal(out[1], Y[-3])
    src = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    src[-1] = 1
    cuda_lib.gemm_rows_gather(R, D, 2, 1, BF16, out, D, src, None, Y, D)
    assert torch.equal(Y[-1], out[1])


def test_many_tokens_and_slots(cuda_lib):
    """More items than resident blocks, more slots than are in flight at once; twice the same bits."""
    T, top, D, R = 3000, 11, 72, 3000 * 11
    rng = np.random.default_rng(6)
    row, source, n = order(rng, T, top, 0.1)
    dO, Y = torch.randn(T, D, device="cuda"), torch.randn(R, D, device="cuda")
    w = torch.rand(T, top, device="cuda")
    outs = []
    for _ in range(2):
        dY, dw = torch.zeros(R, D, device="cuda"), torch.full((T, top), CANARY, device="cuda")
        cuda_lib.gemm_rows_combine_grad(T, top, D, R, F32, dO, D, F32, Y, D, dev(row), w, dY, D, dw)
        outs.append((dY, dw))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    r = torch.from_numpy(row).cuda()
    live = r >= 0
    terms = dO.double()[:, None] * Y.double()[r.clamp_min(0)]
    want = torch.where(live, terms.sum(2), torch.zeros(()).cuda().double())
    assert ((dw.double() - want).abs() <= (D + 1) * U * terms.abs().sum(2)).all()
    moved = torch.zeros(R, D, dtype=torch.float64, device="cuda")
    moved[r[live]] = (w.double()[..., None] * dO.double()[:, None])[live]
    assert ((dY.double() - moved).abs() <= U * moved.abs()).all()


@pytest.mark.parametrize("D", [1, 5, 9, 1001, 2059])
@pytest.mark.parametrize("y_dtype,out", [(F32, F32), (F32, BF16), (F16, F32), (F16, F16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("out_pad", [None, 0])
def test_aligned_rows_that_end_inside_a_piece(cuda_lib, D, y_dtype, out, out_pad):
    """D of no whole 16-byte pieces in rows whose pitch is; outputs of such rows, and of rows at any element."""
    rng = np.random.default_rng(D)
    T, top = 41, 3
    R, pitch = T * top, (D + 7) // 8 * 8
    row, source, n = order(rng, T, top, 0.2)
    w = torch.from_numpy(rng.standard_normal((T, top))).float()
    Y, yv = rows(rng, R, D, y_dtype, pitch - D)
    ldo = pitch if out_pad is None else D
    for beta in (0.0, 0.5):
        o = blank(T, D, out, ldo - D)
        o0 = torch.from_numpy(rng.standard_normal((T, D))).to(DT[out])
        o[1:T + 1, :D] = o0.cuda() if beta else float("nan")
        cuda_lib.gemm_rows_combine(T, top, D, R, y_dtype, Y, pitch, dev(row), w.cuda(), beta, out, o[1:], ldo)
        want, size = orr.combine_reference(yv, row, w.double().numpy(), beta, o0.double().numpy())
        assert (np.abs(inside(o, T, D) - want) <= (top + 2) * U * size + HALF[out] * np.abs(want) + 2.0 ** -25).all()
    if out != y_dtype and out != F32:
        return
    # the incoming gradient in `out`, the rows in y_dtype; and the tokens gathered
    X, xv = rows(rng, T, D, out, pitch - D)
    dY, dw = blank(R, D, y_dtype, ldo - D), torch.empty(T, top, device="cuda")
    cuda_lib.gemm_rows_combine_grad(T, top, D, R, out, X, pitch, y_dtype, Y, pitch, dev(row), w.cuda(), dY[1:], ldo, dw)
    live = row >= 0
    moved = (w.double().numpy()[..., None] * xv[:, None])[live]
    got = inside(dY, R, D)
    assert (np.abs(got[row[live]] - moved) <= (U + HALF[y_dtype]) * np.abs(moved) + 2.0 ** -25).all()
    assert (got[n:] == CANARY).all()
    terms = np.repeat(xv[:, None], top, 1)[live] * yv[row[live]]
    assert (np.abs(dw.cpu().numpy()[live] - terms.sum(1)) <= (D + 1) * U * np.abs(terms).sum(1)).all()
    g = blank(R, D, out, ldo - D)
    cuda_lib.gemm_rows_gather(R, D, T, top, out, X, pitch, dev(source), None, g[1:], ldo)
    got = inside(g, R, D)
    np.testing.assert_array_equal(got[:n], xv[source[:n] // top])
    assert (got[n:] == CANARY).all()


@pytest.mark.parametrize("T,top,D", [(1, 1, 70001), (2, 4, 6644), (3, 1, 31), (216, 4, 6931), (1, 3, 100008), (700, 2, 1000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_gather_of_few_long_rows(cuda_lib, T, top, D, dtype, pad, shift):
    """Rows that several warps share: every element, the ends of the parts and of the rows, nothing beside them."""
    test_gather(cuda_lib, T, top, D, dtype, pad, shift)
