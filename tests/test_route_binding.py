"""The Python binding of the block-scaled rows, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import dense_gemm_epilogues_tcgen05_gb300 as g
    return g


def test_gathered_quantisation_wants_the_rows_of_x(g):
    """Ten rows named out of a hundred: M in the place of X's rows would leave those past the tenth as they were."""
    with pytest.raises(TypeError, match="rows_x"):
        g.gemm_mx_quantize(10, 64, g.MX_E2M1, g.BF16, 1 << 20, 64, 1 << 20, 64, 1 << 20, 2, source=1 << 20, top=1, stream=1)
    assert g.gemm_mx_quantize(0, 64, g.MX_E2M1, g.BF16, 1 << 20, 64, 1 << 20, 64, 1 << 20, 2, stream=1) == 0
    assert g.gemm_mx_quantize(0, 64, g.MX_E2M1, g.BF16, 1 << 20, 64, 1 << 20, 64, 1 << 20, 2, source=1 << 20, top=1, rows_x=100,
                              stream=1) == 0
