"""Arrays that do not start at a multiple of their element's size: refused by the grouped and 8-bit entry points before
any CUDA call (the kernels access whole elements, which the GPU answers with a fault); read as an int address here."""
import pytest

from test_grouped_host import BF16, F16, F32, MISALIGNED, P, g, grouped, i8, quantize, wgrad  # noqa: F401


@pytest.mark.parametrize("call,kw", [
    (grouped, dict(C=P + 1)), (grouped, dict(C=P + 2, c_dtype=F32)), (grouped, dict(A=P + 1)), (grouped, dict(B=P + 1)),
    (grouped, dict(A=P + 2, ab_dtype=F32, c_dtype=F32)), (grouped, dict(bias=P + 2, epilogue=1)),
    (grouped, dict(row_scale=P + 2)), (grouped, dict(offsets=P + 3)),
    (grouped, dict(C=P + 1, K=0)), (grouped, dict(bias=P + 1, epilogue=4, alpha=0.0)),
    (wgrad, dict(C=P + 2)), (wgrad, dict(C=P + 1, c_dtype=F16)), (wgrad, dict(A=P + 1)), (wgrad, dict(D=P + 1)),
    (wgrad, dict(a_sum=P + 2)), (wgrad, dict(offsets=P + 2)), (wgrad, dict(C=P + 2, T=0)),
    (i8, dict(C=P + 1)), (i8, dict(C=P + 2, c_dtype=F32)), (i8, dict(x_scale=P + 2)), (i8, dict(w_scale=P + 1)),
    (i8, dict(bias=P + 2, epilogue=1)), (i8, dict(offsets=P + 2)),
    (quantize, dict(X=P + 1)), (quantize, dict(X=P + 2, x_dtype=F32)), (quantize, dict(scale=P + 2)),
])
def test_refused(g, call, kw):  # noqa: F811
    with pytest.raises(g.GemmError) as e:
        call(g, **kw)
    assert e.value.status == MISALIGNED


@pytest.mark.parametrize("call,kw", [
    (grouped, dict(bias=P + 1)), (grouped, dict(A=P + 1, K=0)), (grouped, dict(row_scale=P + 1, alpha=0.0)),
    (wgrad, dict(A=P + 1, alpha=0.0)), (i8, dict(X=P + 1)), (i8, dict(W=P + 3)), (i8, dict(x_scale=P + 1, K=0)),
    (quantize, dict(Q=P + 1)), (quantize, dict(X=P + 1, K=0, x_dtype=F32)),
])
def test_not_an_alignment_error(g, call, kw):  # noqa: F811
    """What is not read, and codes at any byte: without a GPU these end at a CUDA call or at the range check."""
    with pytest.raises(g.GemmError) as e:
        call(g, **kw)
    assert e.value.status != MISALIGNED
