"""The grouped and 8-bit entry points without a GPU: refusals (all decided before any CUDA call), no-ops,
and the float64 references against brute force."""
import numpy as np
import pytest

from oracle import grouped as og

F32, F16, BF16, E4M3 = range(4)
P = 1 << 20  # an address that is never read: each call is refused or has nothing to do


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import dense_gemm_epilogues_tcgen05_gb300 as g
    return g


def grouped(g, **kw):
    a = dict(G=2, M=8, N=16, K=32, ab_dtype=BF16, offsets=P, A=P, a_stride_m=32, a_stride_k=1, B=P, b_stride_g=512,
             b_stride_k=1, b_stride_n=32, C=P, ldc=16, c_dtype=BF16, alpha=1.0, beta=0.0, bias=None, epilogue=0,
             stream=1)
    a.update(kw)
    return g.gemm_grouped(**a)


def wgrad(g, **kw):
    a = dict(G=2, T=8, M=16, N=32, ab_dtype=BF16, offsets=P, A=P, a_stride_r=16, a_stride_m=1, D=P, d_stride_r=32,
             d_stride_n=1, C=P, c_stride_g=512, ldc=32, c_dtype=F32, alpha=1.0, beta=0.0, a_sum=None, stream=1)
    a.update(kw)
    return g.gemm_grouped_wgrad(**a)


def i8(g, **kw):
    a = dict(G=2, M=8, N=16, K=32, offsets=P, X=P, ldx=32, x_scale=P, W=P, w_stride_g=512, ldw=32, w_scale=P, C=P,
             ldc=16, c_dtype=BF16, alpha=1.0, beta=0.0, bias=None, epilogue=0, stream=1)
    a.update(kw)
    return g.gemm_i8_grouped(**a)


def quantize(g, **kw):
    a = dict(M=8, K=32, x_dtype=BF16, X=P, ldx=32, Q=P, ldq=32, scale=P, stream=1)
    a.update(kw)
    return g.gemm_i8_quantize(**a)


INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3


@pytest.mark.parametrize("call,kw,status", [
    (grouped, dict(G=-1), INVALID), (grouped, dict(M=-1), INVALID), (grouped, dict(K=-1), INVALID),
    (grouped, dict(ldc=15), INVALID), (grouped, dict(C=None), INVALID), (grouped, dict(A=None), INVALID),
    (grouped, dict(B=None), INVALID), (grouped, dict(offsets=None), INVALID), (grouped, dict(epilogue=1), INVALID),
    (grouped, dict(epilogue=6), INVALID), (grouped, dict(epilogue=-1), INVALID), (grouped, dict(b_stride_g=-1), INVALID),
    (grouped, dict(a_stride_m=-4), INVALID), (grouped, dict(ab_dtype=9), INVALID), (grouped, dict(c_dtype=7), INVALID),
    (grouped, dict(ab_dtype=E4M3), UNSUPPORTED), (grouped, dict(c_dtype=E4M3), UNSUPPORTED),
    (grouped, dict(ab_dtype=F32), UNSUPPORTED), (grouped, dict(G=1025), UNSUPPORTED),
    (grouped, dict(M=1 << 31), UNSUPPORTED), (grouped, dict(offsets=P + 2), MISALIGNED),
    (wgrad, dict(T=-1), INVALID), (wgrad, dict(ldc=31), INVALID), (wgrad, dict(c_stride_g=511), INVALID),
    (wgrad, dict(c_stride_g=-512), INVALID), (wgrad, dict(A=None), INVALID), (wgrad, dict(D=None), INVALID),
    (wgrad, dict(C=None), INVALID), (wgrad, dict(offsets=None), INVALID), (wgrad, dict(d_stride_r=-1), INVALID),
    (wgrad, dict(ab_dtype=E4M3), UNSUPPORTED), (wgrad, dict(ab_dtype=F32, c_dtype=F16), UNSUPPORTED),
    (wgrad, dict(G=1025, c_stride_g=512), UNSUPPORTED), (wgrad, dict(a_sum=P + 1), MISALIGNED),
    (wgrad, dict(ldc=1 << 62, M=1 << 30), INVALID),
    (i8, dict(ldx=31), INVALID), (i8, dict(ldw=31), INVALID), (i8, dict(X=None), INVALID), (i8, dict(W=None), INVALID),
    (i8, dict(offsets=None), INVALID), (i8, dict(w_stride_g=-1), INVALID), (i8, dict(c_dtype=E4M3), UNSUPPORTED),
    (i8, dict(K=131072, ldx=131072, ldw=131072), UNSUPPORTED), (i8, dict(epilogue=3), INVALID),
    (i8, dict(G=2000), UNSUPPORTED), (i8, dict(offsets=P + 1), MISALIGNED),
    (quantize, dict(ldx=31), INVALID), (quantize, dict(ldq=31), INVALID), (quantize, dict(scale=None), INVALID),
    (quantize, dict(X=None), INVALID), (quantize, dict(x_dtype=E4M3), UNSUPPORTED), (quantize, dict(x_dtype=5), INVALID),
    (quantize, dict(M=-1), INVALID), (quantize, dict(M=1 << 31), UNSUPPORTED),
])
def test_refusals(g, call, kw, status):
    with pytest.raises(g.GemmError) as e:
        call(g, **kw)
    assert e.value.status == status


def test_nothing_to_do(g):
    assert grouped(g, M=0) == 0 and grouped(g, N=0, ldc=0) == 0 and grouped(g, G=0) == 0
    assert wgrad(g, M=0) == 0 and wgrad(g, N=0) == 0 and wgrad(g, G=0) == 0
    assert i8(g, M=0) == 0 and i8(g, N=0) == 0 and quantize(g, M=0) == 0


def test_references_by_brute_force():
    """Small cases element by element, and planted mistakes that the comparison must see."""
    rng = np.random.default_rng(0)
    off = [0, 2, 2, 5]
    A, B = rng.integers(-3, 4, (5, 4)).astype(float), rng.integers(-3, 4, (3, 4, 3)).astype(float)
    C, bias = rng.integers(-3, 4, (5, 3)).astype(float), rng.integers(-3, 4, (3, 3)).astype(float)
    rs, cs = np.array([1, 2, 0.5, 4, 1]), np.array([[1, 2, 4], [1, 1, 1], [0.5, 2, 1]])
    Y, D = og.grouped_reference(off, A, B, 5, 2.0, 0.5, C, bias, rs, cs)
    for r, e in enumerate([0, 0, 2, 2, 2]):
        for j in range(3):
            z = 2 * rs[r] * cs[e, j] * sum(A[r, k] * B[e, k, j] for k in range(4)) + 0.5 * C[r, j] + bias[e, j]
            assert Y[r, j] == max(z, 0.0) and D[r, j] >= abs(z)
    wrong, _ = og.grouped_reference([0, 3, 3, 5], A, B, 5, 2.0, 0.5, C, bias, rs, cs)
    assert not np.array_equal(wrong, Y)  # one row sent to the wrong expert
    W, _, S, _ = og.wgrad_reference(off, A, C, 2.0, 1.0, np.ones((3, 4, 3)), np.ones((3, 4)))
    for e in range(3):
        for m in range(4):
            assert S[e, m] == 1 + 2 * sum(A[r, m] for r in range(off[e], off[e + 1]))
            for n in range(3):
                assert W[e, m, n] == 1 + 2 * sum(A[r, m] * C[r, n] for r in range(off[e], off[e + 1]))
    q, s = og.quantize_reference(np.array([[254.0, 1.0, 3.0, -5.0], [0, 0, 0, 0], [1.0, np.inf, 0, 0]]))
    assert q.tolist() == [[127, 0, 2, -2], [0, 0, 0, 0], [0, 0, 0, 0]] and s[0] == 2 and s[1] == 0 and np.isnan(s[2])
