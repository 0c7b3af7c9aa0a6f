"""GPU tests of what callers of the mixture-of-experts example give it, beside its plain use."""
import os
import sys

import pytest
import torch

from conftest import REPO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe(cuda_lib):
    sys.path.insert(0, os.path.join(REPO, "examples"))
    import moe_layer
    return moe_layer


def tokens_of(T, D, seed):
    return torch.randn(T, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("T", [1, 45])
def test_8_bit_serving_of_rows_as_callers_have_them(moe, T):
    """Inputs with a pitch, transposed, broadcast, a lone row of an odd stride: what their contiguous copies give."""
    D = 256
    layer = moe.MoeLayer(D, 192, 16, 4)
    layer.quantize()
    x = tokens_of(T, D, 7)
    want = layer.forward_i8(x)
    wide = torch.full((T, D + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + D] = x
    forms = [wide[:, 8:8 + D], x.t().contiguous().t(), x.repeat(1, 2)[:, D:]]
    if T == 1:
        forms.append(x.as_strided((1, D), (1, 1)))
    for xi in forms:
        assert torch.equal(layer.forward_i8(xi), want)
    assert torch.equal(layer.forward_i8(x[:1].expand(T, D)), layer.forward_i8(x[:1].repeat(T, 1)))
    assert moe.g.gemm_device_status() == 0


@pytest.mark.parametrize("what", ["router", "token"])
def test_softmax_scores_of_nan_are_not_hidden(moe, what):
    """A router with a NaN in one expert's weights gives every token NaN scores, a token with an infinity its own: NaN
    in their outputs on every path, and the other tokens' outputs those without it."""
    T, D = 40, 256
    layer = moe.MoeLayer(D, 192, 16, 4)
    layer.quantize()
    layer.quantize_mx()
    x, dy = tokens_of(T, D, 11), tokens_of(T, D, 12)

    def run():
        return [layer.forward(x), layer.forward_i8(x), layer.forward_mx(x), layer.train_step(x, dy)[0], layer.reference(x)]

    want = run()
    bad = torch.ones(T, dtype=torch.bool, device="cuda")
    if what == "router":
        layer.router[3, 5] = float("nan")
    else:
        bad[4:] = False
        x[:4, 7] = float("inf")
    for got, w in zip(run(), want):
        assert got[bad].isnan().all()
        assert moe.relative(got[~bad], w[~bad]) < 1e-3 if what == "token" else True
    assert moe.g.gemm_device_status() == 0


def test_more_experts_a_token_than_the_routing_call_takes(moe):
    """48 of 64 experts: bounds of the example's tests (bf16 1.6e-2, 8 bits 4e-2, 4 bits 1/3)."""
    T, D = 21, 256
    layer = moe.MoeLayer(D, 192, 64, 48)
    layer.quantize()
    layer.quantize_mx()
    x, dy = tokens_of(T, D, 13), tokens_of(T, D, 14)
    want, leaf = layer.reference(x, requires_grad=True)
    want.backward(dy.float())
    out, grads = layer.train_step(x, dy)
    for got, bound in ((layer.forward(x), 1.6e-2), (layer.forward_i8(x), 4e-2), (layer.forward_mx(x), 1 / 3), (out, 1.6e-2)):
        assert moe.relative(got, want) < bound
    for (name, grad), t in zip(grads.items(), leaf):
        assert moe.relative(grad, t.grad) < 1.6e-2, name
    with pytest.raises(moe.g.GemmError):
        layer.train_step(x, dy, router=True)
    x[3, 0] = float("nan")
    offsets, _, weight = layer.route(x)
    assert int(offsets[-1]) == 20 * 48 and not weight[:20 * 48].isnan().any()
    got = layer.forward(x)
    assert got[3].isnan().all() and moe.relative(got[4:], want[4:]) < 1.6e-2
    assert moe.g.gemm_device_status() == 0


@pytest.mark.parametrize("options,paths", [("--d 256 --f 192 --experts 8 --top 2", 3), ("--d 48 --f 80 --experts 8 --top 2", 2),
                                           ("--d 64 --f 64 --experts 40 --top 36", 3)])
def test_the_command(moe, monkeypatch, capsys, options, paths):
    """Widths that are multiples of 16 and not of 32 (no 4-bit products), more experts a token than the routing call
    takes (no router gradient)."""
    monkeypatch.setattr(sys, "argv", ["moe_layer.py", "--tokens", "50", *options.split()])
    moe.main()
    out = capsys.readouterr().out
    assert out.count("serving") == 2 * paths and out.count("training, d") == (4 if "36" in options else 5)


def test_the_reference_does_not_use_the_library(moe, monkeypatch):
    """What the paths are compared with is computed without them."""
    layer = moe.MoeLayer(64, 64, 8, 2)
    x = tokens_of(9, 64, 15)
    want = layer.reference(x)
    for name in [n for n in moe.g.__all__ if n.startswith("gemm")]:
        monkeypatch.setattr(moe.g, name, None)
    again, leaf = layer.reference(x, requires_grad=True, router=True)
    assert moe.relative(again, want) < 1e-5 and len(leaf) == 5
