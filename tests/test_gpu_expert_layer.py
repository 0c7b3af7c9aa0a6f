"""Routing, the movement of rows, quantisation and the grouped products run together, as a layer uses them: each step
against plain operations on that step's own inputs, whole layers captured into graphs and on other streams, and the
example's 4-bit path and router gradient."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle.mx_rows as om
import oracle.route as orr
from conftest import REPO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe(cuda_lib):
    sys.path.insert(0, os.path.join(REPO, "examples"))
    import moe_layer
    return moe_layer


def tokens_of(T, D, seed):
    return torch.randn(T, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16()


def codes_of(q, s, k):
    """Element codes, one per element, and scales."""
    q, s = q.cpu().numpy()[:, :k // 2], s.cpu().numpy()[:, :k // 32]
    return np.stack([q & 15, q >> 4], 2).reshape(q.shape[0], k), s


@pytest.mark.parametrize("T,E,top,dropped", [(1, 8, 2, 0), (37, 16, 4, 5), (300, 64, 6, 40)])
def test_each_step_of_a_4_bit_layer(cuda_lib, moe, T, E, top, dropped):
    """From logits to the output; some tokens are padding (logits of -infinity) and come out as zeros."""
    g, D, F = cuda_lib, 256, 192
    layer = moe.MoeLayer(D, F, E, top)
    layer.quantize_mx()
    x = tokens_of(T, D, T)
    logits = x.float() @ layer.router.t()
    logits[:dropped] = -float("inf")
    expert = torch.empty(T, top, dtype=torch.int32, device="cuda")
    weight = torch.empty(T, top, device="cuda")
    g.gemm_route(T, E, top, g.F32, logits, E, expert, weight, score=g.SCORE_SIGMOID)
    want_e, want_w = orr.route_reference(logits.cpu().double().numpy(), top, orr.SIGMOID)
    np.testing.assert_array_equal(expert.cpu().numpy(), want_e)
    np.testing.assert_allclose(weight.cpu().numpy(), want_w, rtol=(48 + 4 * 10) * U)
    offsets, row, source = layer.sort(expert)
    want = orr.rows_reference(want_e, E)
    for got, w in zip((offsets, row, source), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    rows, live = T * top, int(want[0][-1])
    # codes of the gathered rows; those behind the last stay what the allocation held
    qx, sx = moe.quantize_mx_rows(x, source, top)
    xc, xs = om.quantize_reference(x.cpu().double().numpy(), om.E2M1)
    tok = want[2][:live] // top
    c, s = codes_of(qx[:live], sx[:live], D)
    np.testing.assert_array_equal(c, xc[tok])
    np.testing.assert_array_equal(s, xs[tok])
    h = torch.full((rows, F), 9.0, dtype=torch.bfloat16, device="cuda")
    layer._mx_product((qx, sx), (layer.m1, layer.ms1), offsets, D, layer.b1, g.EPI_BIAS_SILU, h)
    assert (h[live:] == 9.0).all(), "rows behind the last one were written"
    w1 = om.values_of(*codes_of(layer.m1, layer.ms1, D), om.E2M1).reshape(E, F, D)
    z = np.zeros((live, F))
    size = np.zeros((live, F))
    xv, b1 = om.values_of(c, s, om.E2M1), layer.b1.cpu().double().numpy()
    for e in range(E):
        r = slice(want[0][e], want[0][e + 1])
        z[r] = xv[r] @ w1[e].T + b1[e]
        size[r] = np.abs(xv[r]) @ np.abs(w1[e]).T + np.abs(b1[e])
    hv = h[:live].cpu().double().numpy()
    silu = z / (1 + np.exp(-z))
    # one rounding to bf16, fp32 sums (4 matrix instructions) and the activation's slope of at most 1.1
    assert (np.abs(hv - silu) <= 2.0 ** -8 * np.abs(silu) + (5 * 2.0 ** -23 + 5e-7) * 1.1 * size).all()
    y = torch.full((rows, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer._mx_product(moe.quantize_mx_rows(h), (layer.m2, layer.ms2), offsets, F, None, g.EPI_NONE, y)
    out = layer.combine(y, row, weight)
    want_out, terms = orr.combine_reference(y.cpu().double().numpy(), want[1], weight.cpu().double().numpy())
    assert (np.abs(out.cpu().numpy() - want_out) <= (top + 2) * U * terms).all()
    assert (out[:dropped] == 0).all() and g.gemm_device_status() == 0


def test_the_example_in_4_bits_and_its_router_gradient(moe):
    """forward_mx is those steps; its codes hold values to half a step, at most 1/4 of them (1/3 of a value that
    saturates): 2-norm errors of the four quantised operands stay below 1/6 each, in quadrature 1/3.  The router's
    gradient against autograd, through bf16 rows: as the example's other gradients (4 roundings of 2^-8)."""
    T, E, top, D, F = 200, 16, 4, 256, 192
    layer = moe.MoeLayer(D, F, E, top)
    layer.quantize_mx()
    x, dy = tokens_of(T, D, 1), tokens_of(T, D, 2)
    want, leaf = layer.reference(x, requires_grad=True, router=True)
    want.backward(dy.float())
    assert moe.relative(layer.forward_mx(x), want) < 1 / 3
    out, grads = layer.train_step(x, dy, router=True)
    assert moe.relative(out, want) < 1.6e-2
    assert list(grads) == ["x", "w1", "b1", "w2", "router"]
    for (name, grad), t in zip(grads.items(), leaf):
        assert moe.relative(grad, t.grad) < 1.6e-2, name
    assert moe.g.gemm_device_status() == 0


@pytest.mark.parametrize("T", [1, 45])
def test_rows_and_gradients_as_callers_have_them(moe, T):
    """Inputs with a pitch, transposed, broadcast, a lone row of an odd stride, and an fp32 output gradient: what their
    contiguous bf16 copies give (fp32 values that bf16 holds give the same products)."""
    D = 256
    layer = moe.MoeLayer(D, 192, 16, 4)
    layer.quantize_mx()
    x, dy = tokens_of(T, D, 7), tokens_of(T, D, 8)

    def run(x, dy):
        out, grads = layer.train_step(x, dy)
        return [layer.forward(x), layer.forward_mx(x), out, *grads.values()]

    want = run(x, dy)
    wide = torch.full((T, D + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + D] = x
    forms = [(wide[:, 8:8 + D], dy.float()), (x.t().contiguous().t(), dy.t().contiguous().t()),
             (x, dy.double()), (x.repeat(1, 2)[:, :D], dy.float().repeat(1, 2)[:, D:])]
    if T == 1:
        forms.append((x.as_strided((1, D), (1, 1)), dy.as_strided((1, D), (3, 1))))
    for xi, di in forms:
        assert all(torch.equal(a, b) for a, b in zip(run(xi, di), want))
    same = dy[:1].expand(T, D)
    assert all(torch.equal(a, b) for a, b in zip(run(x[:1].expand(T, D), same),
                                                 run(x[:1].repeat(T, 1), same.contiguous())))
    assert moe.g.gemm_device_status() == 0


def test_tokens_of_nan(moe):
    """A token with a NaN has NaN logits and no expert: its output is NaN on every path, the other tokens' outputs and
    the weights' gradients are those without it (bounds of the example's tests; fp32 against fp32, four sums of 256
    terms whose roundings reach 256 x 2^-24 = 1.5e-5 each).  Its place behind the last row is no token's."""
    T, D = 50, 256
    layer = moe.MoeLayer(D, 192, 16, 4)
    layer.quantize()
    layer.quantize_mx()
    x, dy = tokens_of(T, D, 9), tokens_of(T, D, 10)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[0, 17, T - 1]] = True
    x[bad, 5] = float("nan")
    offsets, token, weight = layer.route(x)
    assert int(offsets[-1]) == 47 * 4 and (weight[47 * 4:] == 0).all() and int(token.min()) >= 0
    out, grads = layer.train_step(x, dy, router=False)
    outs = [layer.forward(x), layer.forward_i8(x), layer.forward_mx(x), out]
    keep, dkeep = x[~bad].contiguous(), dy[~bad].contiguous()
    want, leaf = layer.reference(keep, requires_grad=True)
    want.backward(dkeep.float())
    for got, bound in zip(outs, (1.6e-2, 4e-2, 1 / 3, 1.6e-2)):
        assert got[bad].isnan().all() and moe.relative(got[~bad], want) < bound
    assert moe.relative(grads["x"][~bad], leaf[0].grad) < 1.6e-2
    for name, t in zip(("w1", "b1", "w2"), leaf[1:]):
        assert moe.relative(grads[name], t.grad) < 1.6e-2, name
    full = layer.reference(x)
    assert full[bad].isnan().all() and moe.relative(full[~bad], want) < 6.2e-5
    assert moe.g.gemm_device_status() == 0


@pytest.mark.parametrize("T", [3, 700])
def test_graphs_and_streams_give_the_same_bits(moe, T):
    """Whole layers captured and replayed on new tokens, two graphs one after the other, beside a copy that no kernel
    precedes; on a side stream; two layers at once on two streams."""
    layers = [moe.MoeLayer(256, 192, 16, 4, seed=s) for s in (0, 1)]
    for layer in layers:
        layer.quantize_mx()
    xs = [tokens_of(T, 256, s) for s in (3, 4)]
    dy = tokens_of(T, 256, 5)

    def run(layer, x):
        out, grads = layer.train_step(x, dy, router=True)
        return [layer.forward(x), layer.forward_mx(x), out, *grads.values()]

    want = [[run(layer, x) for x in xs] for layer in layers]
    torch.cuda.synchronize()
    graphs = []
    for layer in layers:
        static, fresh = torch.empty_like(xs[0]), torch.empty_like(xs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(layer, xs[0])
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            static.copy_(fresh)
            outs = run(layer, static)
        graphs.append((graph, fresh, outs))
    for i in (0, 1, 0):
        for (graph, fresh, outs), by_x in zip(graphs, want):
            fresh.copy_(xs[i])
            graph.replay()
            for a, b in zip(outs, by_x[i]):
                assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in layers]
    got = []
    for s, layer in zip(streams, layers):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([run(layer, xs[0]) for _ in range(3)])
    torch.cuda.synchronize()
    for rounds, by_x in zip(got, want):
        for r in rounds:
            assert all(torch.equal(a, b) for a, b in zip(r, by_x[0]))
    assert moe.g.gemm_device_status() == 0


def test_calls_in_stream_order(cuda_lib):
    """Each kernel is set up while the one before ends: a chain that overwrites its own inputs, many times over,
    between copies and fills of the same arrays."""
    g = cuda_lib
    T, D, top = 64, 512, 2
    X = torch.randn(T, D, device="cuda")
    row = torch.arange(T * top, dtype=torch.int32, device="cuda").flip(0).view(T, top).contiguous()
    source = torch.empty(T * top, dtype=torch.int32, device="cuda")
    source[row.flatten().long()] = torch.arange(T * top, dtype=torch.int32, device="cuda")
    Y, O = torch.empty(T * top, D, device="cuda"), X.clone()
    for i in range(200):
        g.gemm_rows_gather(T * top, D, T, top, g.F32, O, D, source, None, Y, D)
        if i % 3 == 0:
            O.zero_()
        g.gemm_rows_combine(T, top, D, T * top, g.F32, Y, D, row, None, 0.0, g.F32, O, D)
        if i % 5 == 0:
            Y.fill_(float("nan"))
        O.mul_(0.5)
    assert torch.equal(O, X)  # each round doubles and halves: exact
