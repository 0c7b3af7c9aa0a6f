"""The mixture-of-experts example, small: its three paths against plain fp32 operations.

bf16 values carry a relative rounding of at most 2^-8 each; the output passes two roundings in a row (h, y)
and the gradients up to four (z, dr, dh, dz, then their own), independent over many terms, so 2-norm errors
stay below 4 * 2^-8 = 1.6e-2.  8-bit codes add half a step of max / 127 to x, W1, h and W2: for rows of
K normal values the largest is below 4.5 standard deviations, so a step is below 0.036 of one, uniform error
0.036 / sqrt(12) = 1.03e-2 per operand, four operands in quadrature 2.1e-2; the bound is 4e-2.
"""
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


@pytest.mark.parametrize("tokens,experts,top", [(1, 8, 2), (37, 16, 4), (600, 8, 2)])
def test_moe_layer(moe, tokens, experts, top):
    layer = moe.MoeLayer(256, 192, experts, top)
    layer.quantize()
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, 256, device="cuda", generator=gen).bfloat16()
    dy = torch.randn(tokens, 256, device="cuda", generator=gen).bfloat16()
    want, leaf = layer.reference(x, requires_grad=True)
    want.backward(dy.float())
    assert moe.relative(layer.forward(x), want) < 1.6e-2
    assert moe.relative(layer.forward_i8(x), want) < 4e-2
    out, grads = layer.train_step(x, dy)
    assert moe.relative(out, want) < 1.6e-2
    for (name, grad), t in zip(grads.items(), leaf):
        assert moe.relative(grad, t.grad) < 1.6e-2, name
    assert moe.g.gemm_device_status() == 0
