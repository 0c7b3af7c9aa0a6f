"""GPU tests of the routing's 16-byte paths and of warps that take many tokens, against float64 (bounds: those of
test_gpu_route.py; fp16 outputs also to 2^-25, half a step of its subnormals).

Rows are read in 16-byte pieces where bases and pitches are whole ones and a lane holds a piece or more: from 65
experts on in fp32 and from 129 on in 16 bits.
"""
import numpy as np
import pytest
import torch

import oracle.route as orr
from test_gpu_route import BF16, DT, F16, F32, SIGMOID, SOFTMAX, U, check, logits_of, place, reference, route

pytestmark = pytest.mark.gpu

HALF = {F32: 0.0, F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.mark.parametrize("T,E", [(37, 128), (19, 160), (40, 256), (9, 512), (7, 1000), (5, 1024)])
@pytest.mark.parametrize("pad", [0, 16])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_choices_of_aligned_rows(cuda_lib, T, E, pad, score, dtype):
    dev, x = logits_of(T, E, dtype, E + T, pad=pad)
    assert dev.data_ptr() % 16 == 0 and dev.stride(0) * dev.element_size() % 16 == 0
    bias = torch.from_numpy(np.random.default_rng(E).normal(0, 0.2, E)).float()
    for kw in (dict(renormalise=False), dict(renormalise=True), dict(bias=bias), dict(bias=bias, renormalise=False)):
        kw = dict(score=score, scale=2.5, **kw)
        check(x, route(cuda_lib, dev, T, E, 8, dtype, **kw), reference(x, 8, **kw))


@pytest.mark.parametrize("E,groups,top_groups,group_sum", [(256, 8, 4, 2), (160, 8, 3, 2), (512, 1, 1, 1), (64, 4, 2, 2),
                                                           (1024, 32, 4, 2)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_warps_that_alternate_between_decisions(cuda_lib, E, groups, top_groups, group_sum, score, dtype):
    """30000 tokens of 48 kinds in a random order, so that a warp's next token is often decided another way: in fp32,
    among candidates in 64 bits, all in 64 bits (more candidates than lanes), with nothing available."""
    rng = np.random.default_rng(E)
    kinds = rng.normal(0, 1.5, (48, E))
    kinds[10:14] = kinds[0]
    kinds[14:18] = rng.integers(0, 2, (4, E))              # many equal logits
    kinds[18] = 0.25
    kinds[19, :] = -np.inf
    kinds[20, :] = np.nan
    kinds[21, 3:] = -np.inf
    kinds[22:26][rng.random((4, E)) < 0.3] = -np.inf
    kinds[26:30, ::3] = kinds[26:30, :1]
    x = torch.from_numpy(kinds).to(DT[dtype])
    bias = (0.75 - orr.scores(x[0].double().numpy(), score)).astype(np.float32)  # kind 0: equal up to a rounding
    bias[1::7] = bias[0]
    kw = dict(bias=torch.from_numpy(bias), score=score, groups=groups, top_groups=top_groups, group_sum=group_sum,
              scale=1.5)
    want = reference(x.double().numpy(), 8, **kw)
    pick = rng.integers(0, len(kinds), 30000)
    dev = x.cuda()[torch.from_numpy(pick).cuda()].contiguous()
    got = route(cuda_lib, dev, len(pick), E, 8, dtype, **kw)
    check(x.double().numpy(), got, (want[0][pick], want[1][pick]))


@pytest.mark.parametrize("E", [128, 160, 256, 512, 1000, 1024])
@pytest.mark.parametrize("shift,out_pad", [(0, 0), (0, 3), (1, 0), (1, 8)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_gradient_of_aligned_rows(cuda_lib, E, shift, out_pad, score, renormalise, dtype):
    """Read and written in pieces, one of the two, neither; masked logits, a row of them, repeated and absent experts."""
    T, top = 21, 8
    rng = np.random.default_rng(E + shift)
    x = rng.normal(0, 2, (T, E))
    x[rng.random((T, E)) < 0.1] = -np.inf
    x[3] = -np.inf
    xt = torch.from_numpy(x).to(DT[dtype])
    x = xt.double().numpy()
    expert, _ = orr.route_reference(x, top, score)
    expert[rng.random(expert.shape) < 0.1] = -1
    expert[5, 0], expert[6], expert[7, 1], expert[8, 2:5] = E, -1, expert[7, 0], E - 1
    dw = torch.from_numpy(rng.normal(0, 1, (T, top))).float()
    dev = place(xt, shift=shift)
    out = torch.full((T + 2, E + out_pad), 9.0, dtype=DT[dtype], device="cuda")
    rows = out.flatten()[8:][:T * (E + out_pad)]  # (16 bytes or 32 into the allocation)
    cuda_lib.gemm_route_grad(T, E, top, dtype, dev, dev.stride(0), torch.from_numpy(expert).int().cuda(), dw.cuda(), rows,
                             E + out_pad, score, renormalise, 2.5)
    want, size = orr.route_grad_reference(x, expert, dw.numpy(), score, renormalise, 2.5)
    got = rows.view(T, E + out_pad).cpu().double().numpy()
    assert (got[:, E:] == 9.0).all()
    assert (out.flatten()[:8] == 9.0).all() and (out.flatten()[8 + T * (E + out_pad):] == 9.0).all()
    fin = np.abs(x[np.isfinite(x)]).max()
    sub = 2.0 ** -25 if dtype == F16 else 2.0 ** -120
    assert (np.abs(got[:, :E] - want) <= (3 * (48 + 4 * fin) + 33) * U * size + HALF[dtype] * np.abs(want) + sub).all()


@pytest.mark.parametrize("E", [160, 256, 512])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_gradient_of_many_aligned_tokens(cuda_lib, E, dtype):
    """Several tokens to a warp, up to 256 experts the next one's arrays on their way; the same bits on every call."""
    T, top = 20003, 8
    dev, _ = logits_of(T, E, dtype, 2)
    expert = torch.topk(dev.float(), top).indices.int()
    expert[::5, 2] = -1
    dw = torch.randn(T, top, device="cuda", generator=torch.Generator(device="cuda").manual_seed(E))
    outs = []
    for _ in range(3):
        out = torch.empty(T, E, dtype=DT[dtype], device="cuda")
        cuda_lib.gemm_route_grad(T, E, top, dtype, dev, E, expert, dw, out, E, SOFTMAX, False, 1.0)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    p = torch.softmax(dev.double(), 1)
    d = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
    d = d.scatter_(1, torch.where(expert < 0, E, expert).long(), dw.double())[:, :E]
    want = p * (d - (d * p).sum(1, keepdim=True))
    size = p * (d.abs() + (d * p).abs().sum(1, keepdim=True))
    sub = 2.0 ** -25 if dtype == F16 else 2.0 ** -120
    fin = float(dev.abs().max())
    assert ((out.double() - want).abs() <= (3 * (48 + 4 * fin) + 33) * U * size + HALF[dtype] * want.abs() + sub).all()
