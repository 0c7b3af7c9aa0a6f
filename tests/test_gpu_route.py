"""GPU tests of the routing to experts (gemm_route, gemm_route_grad, gemm_route_rows) against float64.

Choices are equal to the reference's.  Weights: an exponential is within 2 units in the last place (4 u, u =
2^-24), twice for a quotient of two; the rounding of an argument x - m moves it by |x - m| u, twice; the sum has at
most 37 additions in a row; quotient, scale and reciprocal three roundings.  With |x - m| <= 2 max|x| in these
cases (logits masked to the lowest value aside, whose exponentials are 0): (8 + 4 max|x| + 40) u, relative.
Gradients: the same, three times (weight, slope, mean) and at most 33 more additions, of the sum of absolute
terms; and half a unit in the last place of a 16-bit output.
"""
import numpy as np
import pytest
import torch

import oracle.route as orr

pytestmark = pytest.mark.gpu

F32, F16, BF16 = 0, 1, 2
DT = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
U = 2.0 ** -24
SOFTMAX, SIGMOID = 0, 1
LOWEST = float(np.finfo(np.float32).min)


def logits_of(T, E, dtype, seed, std=2.0, pad=0, shift=0):
    """Rounded logits: device rows of pitch E + pad that begin `shift` elements into their allocation."""
    x = torch.from_numpy(np.random.default_rng(seed).normal(0, std, (T, E))).to(DT[dtype])
    return place(x, pad, shift), x.double().numpy()


def place(x, pad=0, shift=0):
    T, E = x.shape
    buf = torch.full((shift + T * (E + pad),), float("nan"), dtype=x.dtype)
    rows = buf[shift:].view(T, E + pad)
    rows[:, :E] = x
    return buf.cuda()[shift:].view(T, E + pad)


def route(g, dev, T, E, top, dtype, **kw):
    """expert, weight from buffers with a guard on both sides."""
    e = torch.full((T * top + 16,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T * top + 16,), -7.0, device="cuda")
    bias = kw.pop("bias", None)
    g.gemm_route(T, E, top, dtype, dev, dev.stride(0), e[8:], w[8:], None if bias is None else bias.cuda(), **kw)
    torch.cuda.synchronize()
    for t in (e, w):
        assert (t[:8] == -7).all() and (t[8 + T * top:] == -7).all()
    return e[8:8 + T * top].view(T, top).cpu().numpy(), w[8:8 + T * top].view(T, top).cpu().double().numpy()


def reference(x, top, bias=None, score=SOFTMAX, groups=1, top_groups=1, group_sum=1, renormalise=True, scale=1.0):
    return orr.route_reference(x, top, score, None if bias is None else bias.double().numpy(), groups, top_groups,
                               group_sum, renormalise, scale)


def check(x, got, want):
    np.testing.assert_array_equal(got[0], want[0])
    fin = x[np.isfinite(x) & (np.abs(x) < 1e30)]
    rel = (48 + 4 * (np.abs(fin).max() if fin.size else 0)) * U
    assert (np.abs(got[1] - want[1]) <= rel * np.abs(want[1]) + 2.0 ** -140).all()


@pytest.mark.parametrize("T,E", [(1, 1), (1, 8), (5, 31), (64, 32), (33, 60), (7, 64), (130, 128), (9, 160), (40, 256),
                                 (11, 257), (6, 512), (5, 700), (3, 1024)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_plain_choices(cuda_lib, T, E, score, dtype):
    """Every width of a lane, odd numbers of experts, rows that 16-byte loads cannot read; ties of 16-bit logits."""
    dev, x = logits_of(T, E, dtype, E + T, pad=E % 3, shift=E % 2)
    top = min(E, 1 + E % 9)
    for renormalise in (False, True):
        kw = dict(score=score, renormalise=renormalise, scale=2.5)
        check(x, route(cuda_lib, dev, T, E, top, dtype, **kw), reference(x, top, **kw))


@pytest.mark.parametrize("E,groups,top_groups", [(256, 8, 4), (64, 4, 1), (128, 16, 3), (160, 8, 3), (60, 5, 5),
                                                 (32, 32, 7), (1024, 32, 4), (96, 3, 2), (8, 8, 2), (1024, 2, 1)])
@pytest.mark.parametrize("group_sum", [1, 2])
@pytest.mark.parametrize("bias", [False, True])
def test_groups(cuda_lib, E, groups, top_groups, group_sum, bias):
    T, top = 23, min(8, E)
    dev, x = logits_of(T, E, F32, E + groups)
    b = torch.from_numpy(np.random.default_rng(E).normal(0, 0.2, E)).float() if bias else None
    for score in (SOFTMAX, SIGMOID):
        kw = dict(bias=b, score=score, groups=groups, top_groups=top_groups, group_sum=group_sum, scale=1.5)
        check(x, route(cuda_lib, dev, T, E, top, F32, **kw), reference(x, top, **kw))


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("E,groups", [(64, 1), (256, 8), (160, 8)])
def test_neighbours_closer_than_fp32(cuda_lib, score, E, groups):
    """Selection scores that differ by less than fp32 scores are exact, and equal ones: decided as in 64 bits.  Of two
    experts with logits a and b, biases make the scores equal to within one fp32 rounding of the bias."""
    rng = np.random.default_rng(E + groups)
    T = 64
    xv = rng.normal(0, 1, (T, E)).astype(np.float32)
    xv[: T // 2] = xv[0]                                 # one row of logits, for which the biases are chosen:
    s = np.stack([orr.scores(r, score) for r in xv[:1]])[0]
    b = (0.75 - s).astype(np.float32)                    # scores + bias all 0.75, up to the bias's rounding
    b[::5] = b[0]
    xv[T // 2:, ::3] = xv[T // 2:, :1]                   # equal logits under different and equal biases
    x = xv.astype(np.float64)
    kw = dict(bias=torch.from_numpy(b), score=score, groups=groups, top_groups=max(1, groups // 2),
              group_sum=2 if groups > 1 else 1, renormalise=score == SIGMOID)
    check(x, route(cuda_lib, torch.from_numpy(xv).cuda(), T, E, 8, F32, **kw), reference(x, 8, **kw))


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("groups,group_sum,with_bias", [(1, 1, False), (4, 1, False), (4, 2, False), (1, 1, True), (4, 2, True)])
def test_masks(cuda_lib, score, groups, group_sum, with_bias):
    """Rows of -infinity, NaN and the lowest value, alone and mixed; fewer experts than slots; +infinity; 0 and -0;
    a bias of -infinity, NaN."""
    E, top, inf, nan = 16, 6, np.inf, np.nan
    rng = np.random.default_rng(3)
    rows = [np.full(E, -inf), np.full(E, nan), np.full(E, LOWEST), np.zeros(E), -np.zeros(E)]
    for n in (1, 5, 6, 9):
        r = np.full(E, -inf)
        r[rng.permutation(E)[:n]] = rng.normal(0, 2, n)
        rows += [r, np.where(r == -inf, LOWEST, r), np.where(r == -inf, nan, r)]
    r = rng.normal(0, 1, E)
    for v in (inf, 1e38, -1e38, 95.0, -95.0, -150.0):
        q = r.copy()
        q[[3, 11]] = v
        rows += [q, np.where(np.arange(E) % 8 == 3, v, -inf), np.full(E, v)]
    q = np.where(np.arange(E) % 2 == 0, 0.0, -0.0)
    x = np.stack(rows + [q]).astype(np.float32)
    bias = None
    if with_bias:
        bias = torch.from_numpy(rng.normal(0, 0.3, E)).float()
        bias[2], bias[9] = -inf, nan
    for renormalise in (False, True):
        kw = dict(bias=bias, score=score, groups=groups, top_groups=max(1, groups - 1), group_sum=group_sum,
                  renormalise=renormalise)
        got = route(cuda_lib, torch.from_numpy(x).cuda(), len(x), E, top, F32, **kw)
        want = reference(x.astype(np.float64), top, **kw)
        np.testing.assert_array_equal(got[0], want[0])
        finite = np.where(np.isfinite(x) & (np.abs(x) < 1e30), np.abs(x), 0).max(1, keepdims=True)
        assert (np.abs(got[1] - want[1]) <= (48 + 4 * finite) * U * np.abs(want[1]) + 2.0 ** -126).all()


def test_many_tokens(cuda_lib):
    """More tokens than the grid's warps: each warp takes several."""
    T, E, top = 20011, 64, 6
    dev, x = logits_of(T, E, BF16, 1)
    got = route(cuda_lib, dev, T, E, top, BF16)
    order = np.argsort(-x, axis=1, kind="stable")[:, :top]
    np.testing.assert_array_equal(got[0], order)
    e = np.exp(np.take_along_axis(x, order, 1) - x.max(1, keepdims=True))
    np.testing.assert_allclose(got[1], e / e.sum(1, keepdims=True), rtol=100 * U)


@pytest.mark.parametrize("E,top", [(1, 1), (8, 8), (60, 4), (128, 8), (257, 3), (1024, 32)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient(cuda_lib, E, top, score, renormalise, dtype):
    """Against the formula; experts of -1 and past E, one expert in two slots, masked logits, rows without experts."""
    T = 37
    rng = np.random.default_rng(E + top)
    x = rng.normal(0, 2, (T, E))
    x[rng.random((T, E)) < 0.1] = -np.inf
    x[3] = -np.inf
    xt = torch.from_numpy(x).to(DT[dtype])
    x = xt.double().numpy()
    expert, _ = orr.route_reference(x, top, score)
    expert[rng.random(expert.shape) < 0.1] = -1
    expert[5, 0], expert[6] = E, -1
    if top > 1:
        expert[7, 1] = expert[7, 0]
    dw = torch.from_numpy(rng.normal(0, 1, (T, top))).float()
    dev = place(xt, pad=E % 2, shift=E % 3)
    ldd = E + 5
    out = torch.full((T, ldd), 9.0, dtype=DT[dtype], device="cuda")
    cuda_lib.gemm_route_grad(T, E, top, dtype, dev, dev.stride(0), torch.from_numpy(expert).int().cuda(), dw.cuda(), out,
                             ldd, score, renormalise, 2.5)
    want, size = orr.route_grad_reference(x, expert, dw.numpy(), score, renormalise, 2.5)
    out = out.cpu().double().numpy()
    assert (out[:, E:] == 9.0).all()
    fin = np.abs(x[np.isfinite(x)]).max()
    half = {F32: 0.0, BF16: 2.0 ** -8}[dtype]
    assert (np.abs(out[:, :E] - want) <= (3 * (48 + 4 * fin) + 33) * U * size + half * np.abs(want) + 2.0 ** -120).all()


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_gradient_by_differences(cuda_lib, score):
    """sum(dw * weight) of two calls a step apart, in the direction of each logit; fp32 weights are off by 60 u at
    most, so a quotient over 2 h is off by 60 u (sum of |dw|) / h, and by h^2 / 6 times the third derivative (below 1
    per unit of |dw|)."""
    E, top, h = 12, 4, 2.0 ** -7
    rng = np.random.default_rng(8)
    x, dw = rng.normal(0, 1, E).astype(np.float32), rng.normal(0, 1, top).astype(np.float32)
    x[:top] += 6.0  # the choice survives the steps
    steps = np.concatenate([x + h * np.eye(E), x - h * np.eye(E)]).astype(np.float32)
    for renormalise in (False, True):
        kw = dict(score=score, renormalise=renormalise)
        e, w = route(cuda_lib, torch.from_numpy(steps).cuda(), 2 * E, E, top, F32, **kw)
        slot = np.argsort(e, 1)  # the same experts in another order
        val = (np.take_along_axis(w, slot, 1) * dw).sum(1)
        expert = torch.arange(top, dtype=torch.int32, device="cuda").view(1, top)
        out = torch.empty(1, E, device="cuda")
        cuda_lib.gemm_route_grad(1, E, top, F32, torch.from_numpy(x[None]).cuda(), E, expert, torch.from_numpy(dw).cuda(),
                                 out, E, score, renormalise)
        diff = (val[:E] - val[E:]) / (2 * h)
        bound = np.abs(dw).sum() * (60 * U / h + h * h / 6)
        assert (np.abs(out.cpu().numpy()[0] - diff) <= bound).all()


@pytest.mark.parametrize("T,top,E", [(0, 2, 5), (1, 1, 1), (1, 8, 64), (7, 3, 4), (100, 4, 1024), (512, 8, 64), (513, 8, 64),
                                     (5000, 1, 300), (16384, 8, 256), (30000, 5, 7), (40000, 8, 1000)])
def test_rows(cuda_lib, T, top, E):
    """One block and many; out-of-range experts; all of one expert; the arrays' neighbours untouched."""
    rng = np.random.default_rng(T + E)
    for kind in ("random", "one", "none", "skewed"):
        expert = {"random": lambda: rng.integers(-1, E + 1, (T, top)), "one": lambda: np.full((T, top), E - 1),
                  "none": lambda: np.full((T, top), -1),
                  "skewed": lambda: np.minimum(rng.geometric(0.3, (T, top)) - 1, E - 1)}[kind]()
        if T * top > 100000 and kind != "random":
            continue
        P = T * top
        off = torch.full((E + 1 + 8,), -7, dtype=torch.int32, device="cuda")
        row, src = (torch.full((P + 8,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        need = cuda_lib.gemm_route_rows_workspace_size(T, top, E)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        cuda_lib.gemm_route_rows(T, top, E, torch.from_numpy(expert).int().cuda(), off, row, src, ws, need)
        want = orr.rows_reference(expert, E)
        np.testing.assert_array_equal(off[:E + 1].cpu().numpy(), want[0])
        np.testing.assert_array_equal(row[:P].cpu().numpy(), want[1].reshape(-1))
        np.testing.assert_array_equal(src[:P].cpu().numpy(), want[2])
        assert (off[E + 1:] == -7).all() and (row[P:] == -7).all() and (src[P:] == -7).all()
        cuda_lib.gemm_route_rows(T, top, E, torch.from_numpy(expert).int().cuda(), off, None, src, ws, need)
        np.testing.assert_array_equal(src[:P].cpu().numpy(), want[2])


@pytest.mark.parametrize("E,top", [(8, 20), (3, 32), (40, 32), (64, 31), (256, 32)])
@pytest.mark.parametrize("biased", [False, True])
def test_more_slots_than_experts_or_nearly(cuda_lib, E, top, biased):
    """Slots left over get -1 and weight 0; 31 and 32 slots, which the lanes' maxima cannot bound; equal logits, whose
    candidates are more than the lanes."""
    T = 19
    _, x = logits_of(T, E, F32, E)
    x[5], x[6] = 0.25, np.round(x[6])
    b = torch.from_numpy(np.random.default_rng(top).normal(0, 0.1, E)).float() if biased else None
    if biased:
        x[7] = -1.5  # equal scores but for the bias
    for score in (SOFTMAX, SIGMOID):
        kw = dict(bias=b, score=score, renormalise=True)
        got = route(cuda_lib, torch.from_numpy(x).float().cuda(), T, E, top, F32, **kw)
        check(x, got, reference(x, top, **kw))


def test_all_equal(cuda_lib):
    """A router before training: every logit and bias 0.  The lower indexes, groups among them."""
    T, E, top = 300, 256, 8
    x = torch.zeros(T, E, device="cuda")
    kw = dict(bias=torch.zeros(E), score=SIGMOID, groups=8, top_groups=4, group_sum=2)
    e, w = route(cuda_lib, x, T, E, top, F32, **kw)
    assert (e == np.arange(top)).all() and (w == 0.125).all()


def test_large_biases(cuda_lib):
    """Sums of a group's two that nearly cancel, and biases far above the scores: decided by 64-bit sums."""
    rng = np.random.default_rng(4)
    T, E = 64, 64
    x = rng.normal(0, 1, (T, E)).astype(np.float32)
    b = np.where(rng.random(E) < 0.5, 1000.0, -1000.0) + rng.normal(0, 1e-4, E)
    b = torch.from_numpy(b).float()
    kw = dict(bias=b, score=SIGMOID, groups=16, top_groups=5, group_sum=2)
    check(x.astype(np.float64), route(cuda_lib, torch.from_numpy(x).cuda(), T, E, 6, F32, **kw),
          reference(x.astype(np.float64), 6, **kw))


def test_gradient_of_many_tokens(cuda_lib):
    """More tokens than the grid's warps; the same bits on every call."""
    T, E, top = 20003, 64, 4
    dev, _ = logits_of(T, E, F32, 2)
    expert = torch.topk(dev, top).indices.int()
    dw = torch.randn(T, top, device="cuda")
    outs = []
    for _ in range(3):
        out = torch.empty(T, E, device="cuda")
        cuda_lib.gemm_route_grad(T, E, top, F32, dev, E, expert, dw, out, E, SOFTMAX, False, 1.0)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    p = torch.softmax(dev.double(), 1)
    d = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, expert.long(), dw.double())
    want = p * (d - (d * p).sum(1, keepdim=True))
    size = p * (d.abs() + (d * p).abs().sum(1, keepdim=True))
    assert ((out.double() - want).abs() <= 300 * U * size + 2.0 ** -120).all()
