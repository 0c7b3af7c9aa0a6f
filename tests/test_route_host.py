"""Routing, the movement of rows and the block-scaled rows and experts without a GPU: refusals (all decided before
any CUDA call), no-ops, and the float64 references against brute force and planted mistakes."""
import numpy as np
import pytest

import oracle.mx_rows as om
import oracle.route as orr

F32, F16, BF16, E4M3 = range(4)
P = 1 << 20  # an address that is never read: each call is refused or has nothing to do
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import dense_gemm_epilogues_tcgen05_gb300 as g
    return g


DEFAULTS = {
    "gemm_route": dict(T=4, E=64, top=8, l_dtype=F32, logits=P, ldl=64, expert=P, weight=P, bias=P, score=1, groups=8,
                       top_groups=4, group_sum=2),
    "gemm_route_grad": dict(T=4, E=64, top=8, l_dtype=F32, logits=P, ldl=64, expert=P, dweight=P, dlogits=P, ldd=64),
    "gemm_route_rows": dict(T=4096, top=8, E=64, expert=P, offsets=P, row=P, source=P, workspace=P,
                            workspace_bytes=1 << 20),
    "gemm_rows_gather": dict(R=8, D=64, T=4, top=2, dtype=BF16, X=P, ldx=64, source=P, weight=P, Y=P, ldy=64),
    "gemm_rows_combine": dict(T=4, top=2, D=64, R=8, y_dtype=BF16, Y=P, ldy=64, row=P, weight=P, beta=0.0,
                              out_dtype=BF16, Out=P, ldo=64),
    "gemm_rows_combine_grad": dict(T=4, top=2, D=64, R=8, d_dtype=BF16, dOut=P, ldd=64, y_dtype=BF16, Y=P, ldy=64,
                                   row=P, weight=P, dY=P, lddy=64, dweight=P),
    "gemm_mx_quantize": dict(M=8, K=64, elem=1, x_dtype=BF16, X=P, ldx=64, Q=P, ldq=64, scale=P, lds=2, source=P, top=2,
                             rows_x=4),
    "gemm_mx_dequantize": dict(M=8, K=64, elem=1, Q=P, ldq=64, scale=P, lds=2, y_dtype=BF16, Y=P, ldy=64),
    "gemm_mx_grouped": dict(G=2, M=8, N=16, K=512, elem=1, offsets=P, X=P, ldx=512, x_scale=P, ldxs=16, W=P,
                            w_stride_g=8192, ldw=512, w_scale=P, ws_stride_g=256, ldws=16, C=P, ldc=16, c_dtype=BF16,
                            alpha=1.0, beta=0.0, bias=None, epilogue=0),
}


def call(g, name, **kw):
    a = dict(DEFAULTS[name], stream=1)
    a.update(kw)
    return getattr(g, name)(**a)


BIG = (1 << 30) + 1
REFUSED = [
    ("gemm_route", INVALID, [dict(T=-1), dict(E=0), dict(top=0), dict(l_dtype=7), dict(score=2), dict(score=-1),
                             dict(groups=0), dict(groups=7), dict(top_groups=0), dict(top_groups=9), dict(group_sum=0),
                             dict(group_sum=3), dict(ldl=63), dict(logits=None), dict(expert=None), dict(weight=None)]),
    ("gemm_route", UNSUPPORTED, [dict(l_dtype=E4M3), dict(E=1025, groups=1), dict(top=33), dict(groups=64),
                                 dict(T=BIG // 8 + 1)]),
    ("gemm_route", MISALIGNED, [dict(logits=P + 2), dict(l_dtype=F16, logits=P + 1), dict(bias=P + 2),
                                dict(expert=P + 1), dict(weight=P + 3)]),
    ("gemm_route_grad", INVALID, [dict(T=-1), dict(E=0), dict(top=0), dict(score=5), dict(ldl=63), dict(ldd=63),
                                  dict(logits=None), dict(expert=None), dict(dweight=None), dict(dlogits=None)]),
    ("gemm_route_grad", UNSUPPORTED, [dict(l_dtype=E4M3), dict(E=1025), dict(top=33)]),
    ("gemm_route_grad", MISALIGNED, [dict(dlogits=P + 2), dict(dweight=P + 1)]),
    ("gemm_route_rows", INVALID, [dict(T=-1), dict(top=0), dict(E=0), dict(expert=None), dict(offsets=None),
                                  dict(source=None)]),
    ("gemm_route_rows", UNSUPPORTED, [dict(E=1025), dict(T=BIG // 8 + 1)]),
    ("gemm_route_rows", MISALIGNED, [dict(offsets=P + 2), dict(row=P + 1), dict(expert=P + 2), dict(source=P + 3)]),
    ("gemm_route_rows", WORKSPACE, [dict(workspace=None), dict(workspace_bytes=100), dict(workspace=P + 4)]),
    ("gemm_rows_gather", INVALID, [dict(R=-1), dict(D=-1), dict(top=0), dict(X=None), dict(Y=None), dict(source=None),
                                   dict(ldx=63), dict(ldy=63), dict(dtype=9)]),
    ("gemm_rows_gather", UNSUPPORTED, [dict(dtype=E4M3), dict(D=(1 << 23) + 1), dict(T=BIG), dict(R=1 << 31)]),
    ("gemm_rows_gather", MISALIGNED, [dict(X=P + 1), dict(source=P + 2), dict(weight=P + 1)]),
    ("gemm_rows_combine", INVALID, [dict(T=-1), dict(R=-1), dict(top=0), dict(Out=None), dict(Y=None), dict(row=None),
                                    dict(ldo=63), dict(ldy=63)]),
    ("gemm_rows_combine", UNSUPPORTED, [dict(out_dtype=F16), dict(y_dtype=E4M3), dict(D=(1 << 23) + 1)]),
    ("gemm_rows_combine", MISALIGNED, [dict(Out=P + 1), dict(Y=P + 1), dict(row=P + 2)]),
    ("gemm_rows_combine_grad", INVALID, [dict(T=-1), dict(top=0), dict(dOut=None), dict(Y=None), dict(row=None),
                                         dict(ldd=63), dict(ldy=63), dict(lddy=63)]),
    ("gemm_rows_combine_grad", UNSUPPORTED, [dict(d_dtype=F16), dict(d_dtype=BF16, y_dtype=F32), dict(R=1 << 31)]),
    ("gemm_rows_combine_grad", MISALIGNED, [dict(dY=P + 1), dict(dweight=P + 2), dict(weight=P + 1)]),
    ("gemm_mx_quantize", INVALID, [dict(M=-1), dict(K=48), dict(K=-32), dict(elem=2), dict(x_dtype=8), dict(X=None),
                                   dict(Q=None), dict(scale=None), dict(ldx=63), dict(ldq=63), dict(ldq=65), dict(lds=1),
                                   dict(top=0), dict(rows_x=-1), dict(source=None)]),
    ("gemm_mx_quantize", UNSUPPORTED, [dict(x_dtype=E4M3), dict(M=1 << 31, rows_x=1 << 31)]),
    ("gemm_mx_quantize", MISALIGNED, [dict(X=P + 1), dict(source=P + 2)]),
    ("gemm_mx_dequantize", INVALID, [dict(M=-1), dict(K=33), dict(elem=-1), dict(Y=None), dict(Q=None),
                                     dict(scale=None), dict(ldy=63), dict(ldq=62), dict(lds=1)]),
    ("gemm_mx_dequantize", UNSUPPORTED, [dict(y_dtype=E4M3)]),
    ("gemm_mx_dequantize", MISALIGNED, [dict(Y=P + 1)]),
    ("gemm_mx_grouped", INVALID, [dict(G=-1), dict(M=-1), dict(K=500), dict(elem=3), dict(offsets=None), dict(X=None),
                                  dict(W=None), dict(x_scale=None), dict(w_scale=None), dict(C=None), dict(ldc=15),
                                  dict(ldx=480), dict(ldw=480), dict(ldxs=15), dict(ldws=15), dict(w_stride_g=-2),
                                  dict(w_stride_g=0), dict(ws_stride_g=0), dict(w_stride_g=8193), dict(epilogue=1),
                                  dict(epilogue=9), dict(c_dtype=9)]),
    ("gemm_mx_grouped", UNSUPPORTED, [dict(c_dtype=E4M3), dict(G=1025), dict(M=1 << 31)]),
    ("gemm_mx_grouped", MISALIGNED, [dict(X=P + 8), dict(W=P + 8), dict(x_scale=P + 1), dict(w_scale=P + 4),
                                     dict(ldx=514), dict(ldw=520), dict(ldxs=17), dict(ldws=24), dict(ws_stride_g=264),
                                     dict(w_stride_g=8200), dict(C=P + 1), dict(offsets=P + 2), dict(row_scale=P + 2)]),
]


@pytest.mark.parametrize("name,status,kw", [(n, s, kw) for n, s, many in REFUSED for kw in many], ids=str)
def test_refusals(g, name, status, kw):
    with pytest.raises(g.GemmError) as e:
        call(g, name, **kw)
    assert e.value.status == status


def test_nothing_to_do(g):
    for name, kw in [("gemm_route", dict(T=0)), ("gemm_route_grad", dict(T=0)), ("gemm_rows_gather", dict(R=0)),
                     ("gemm_rows_gather", dict(D=0, ldx=0, ldy=0)), ("gemm_rows_combine", dict(T=0)),
                     ("gemm_rows_combine", dict(D=0)), ("gemm_rows_combine_grad", dict(dY=None, dweight=None)),
                     ("gemm_rows_combine_grad", dict(T=0)), ("gemm_mx_quantize", dict(M=0)),
                     ("gemm_mx_quantize", dict(K=0)), ("gemm_mx_quantize", dict(rows_x=0)),
                     ("gemm_mx_dequantize", dict(M=0)), ("gemm_mx_grouped", dict(M=0)), ("gemm_mx_grouped", dict(G=0)),
                     ("gemm_mx_grouped", dict(N=0, ldc=0))]:
        assert call(g, name, **kw) == 0, name


def test_workspace_size(g):
    assert g.gemm_route_rows_workspace_size(512, 8, 64) == 0  # one block
    assert g.gemm_route_rows_workspace_size(16384, 8, 256) == 128 * 256 * 4
    assert g.gemm_route_rows_workspace_size(1 << 27, 8, 1024) == 144 * 1024 * 4
    assert g.gemm_route_rows_workspace_size(-1, 8, 64) == 0 and g.gemm_route_rows_workspace_size(4096, 8, 2000) == 0


def test_route_reference_by_hand():
    x = np.array([[0.0, 2.0, -1.0, 2.0, np.nan, -np.inf], [-np.inf] * 6, [1.0, np.inf, 0, 0, 0, 0]])
    e, w = orr.route_reference(x, 3, orr.SOFTMAX)
    p = np.exp([2.0, 2.0, 0.0]) / np.exp([2.0, 2.0, 0.0]).sum()
    assert e.tolist() == [[1, 3, 0], [-1, -1, -1], [1, 0, 2]]
    np.testing.assert_allclose(w[0], p, rtol=1e-15)
    assert w[1].tolist() == [0, 0, 0] and w[2].tolist() == [1, 0, 0]
    # a bias moves the choice and not the weight; groups {0, 1, 2}, {3, 4, 5}
    e, w = orr.route_reference(x[:1], 2, orr.SIGMOID, np.array([9.0, 0, 0, 0, 0, 0]), 2, 1, 2, False, 2.0)
    assert e.tolist() == [[0, 1]] and np.allclose(w[0], [1.0, 2 / (1 + np.exp(-2.0))])
    # of two equally worthy groups the lower one
    e, _ = orr.route_reference(np.array([[1.0, 2.0, 2.0, 1.0]]), 1, orr.SOFTMAX, groups=2, top_groups=1)
    assert e.tolist() == [[1]]


@pytest.mark.parametrize("kind", [orr.SOFTMAX, orr.SIGMOID])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_gradient_reference_by_differences(kind, renormalise):
    rng = np.random.default_rng(kind + 2 * renormalise)
    x, dw = rng.standard_normal((2, 7)), rng.standard_normal((2, 3))
    expert, _ = orr.route_reference(x, 3, kind)
    dx, size = orr.route_grad_reference(x, expert, dw, kind, renormalise, 2.5)
    assert (size >= np.abs(dx) - 1e-15).all()
    h = 1e-6
    for t in range(2):
        for e in range(7):
            def loss(d):
                y = x[t].copy()
                y[e] += d
                return float((dw[t] * orr.weights_of(y, expert[t], kind, renormalise, 2.5)).sum())
            assert abs((loss(h) - loss(-h)) / (2 * h) - dx[t, e]) < 1e-8


def test_rows_references_by_hand():
    expert = np.array([[2, 0], [0, -1], [2, 5], [0, 2]])
    off, row, source = orr.rows_reference(expert, 4)
    assert off.tolist() == [0, 3, 3, 6, 6]
    assert row.tolist() == [[3, 0], [1, -1], [4, -1], [2, 5]]
    assert source.tolist() == [1, 2, 6, 0, 4, 7, -1, -1]
    Y = np.arange(12.0).reshape(6, 2)
    out, size = orr.combine_reference(Y, row, np.array([[1, 2], [3, 4], [-1, 1], [0.5, 1]]), 2.0, np.ones((4, 2)))
    assert out.tolist() == [[6 + 0 + 2, 7 + 2 + 2], [6 + 2, 9 + 2], [-8 + 2, -9 + 2], [2 + 10 + 2, 2.5 + 11 + 2]]
    assert size[2].tolist() == [10, 11]


@pytest.mark.parametrize("elem", [om.E4M3, om.E2M1])
def test_quantizer_reference(elem):
    """Against every representable value and midpoint by brute force, the CPU's E4M3 cast, and the input preparation."""
    import torch
    import workloads as wl
    table = om._table(elem)
    mid = (table[1:] + table[:-1]) / 2
    codes = om.nearest_codes(mid, elem)
    assert (codes % 2 == 0).all() and (np.abs(codes - (np.arange(len(mid)) + 0.5)) == 0.5).all()
    assert (om.nearest_codes(-table, elem) == np.arange(len(table)) + (8 if elem == om.E2M1 else 128)).all()
    if elem == om.E4M3:
        v = np.linspace(-460, 460, 4001)
        cast = torch.from_numpy(v).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        np.testing.assert_array_equal(om.nearest_codes(torch.from_numpy(v).float().double().numpy(), elem), cast)
    x = np.random.default_rng(5).standard_normal((8, 96)).astype(np.float32) * 10.0 ** np.arange(-4, 4)[:, None]
    codes, scale = om.quantize_reference(x.astype(np.float64), elem)
    q, s = wl.mx_quantize(torch.from_numpy(x), "e2m1" if elem == om.E2M1 else "e4m3")
    np.testing.assert_array_equal(om.packed(codes, elem), q.numpy())
    np.testing.assert_array_equal(scale, s.numpy())
    # off by one in the scale, or rounding down, is seen
    assert not np.array_equal(om.nearest_codes(x.reshape(8, 3, 32) * np.exp2(126.0 - scale)[..., None], elem).reshape(8, 96), codes)
    y = om.values_of(codes, scale, elem)
    step = {om.E2M1: 1.0, om.E4M3: 32.0}[elem]  # the widest between neighbours; above the largest value, to 2^(emax+1)
    assert (np.abs(y - x) <= np.repeat(np.exp2(scale - 127.0), 32, 1) * max(step, 8.0 - 6.0 if elem == om.E2M1 else 64.0)).all()
