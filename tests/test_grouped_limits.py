"""Sizes next to 2^31 in the grouped and 8-bit entry points, on the CPU: what the kernels' 32-bit indexes cannot hold
is refused before any CUDA call, and what is let through they can round up to a tile."""
import re

import pytest

from conftest import REPO
from test_grouped_host import UNSUPPORTED, g, grouped, i8, wgrad  # noqa: F401 (g is a fixture)

LIMIT = (1 << 31) - 1024


@pytest.mark.parametrize("call,dims", [(grouped, ("M", "N", "K")), (wgrad, ("T", "M", "N")), (i8, ("M", "N"))])
@pytest.mark.parametrize("size", [LIMIT + 1, (1 << 31) - 256, (1 << 31) - 63, (1 << 31) - 1])
def test_refused(g, call, dims, size):  # noqa: F811
    for d in dims:
        kw = {d: size}
        if d == "N":
            kw["ldc"] = size
        if call is wgrad:
            kw["c_stride_g"] = 1 << 60
        with pytest.raises(g.GemmError) as e:
            call(g, **kw)
        assert e.value.status == UNSUPPORTED, kw


def test_limit_is_the_headers(g):  # noqa: F811
    text = open(REPO + "/include/gemm_gb300.h").read()
    assert int(re.search(r"#define GEMM_GROUPED_MAX_EXTENT (\d+)", text).group(1)) == g.GROUPED_MAX_EXTENT == LIMIT


def test_rounding_up_fits():
    """The sums that the kernels form at the limit: the widest stage of k is 4 boxes of 128, tiles are 256 wide, and
    the column sums step by 4 * 128 rows of which the last may begin 128 past the end."""
    for step in (16, 64, 128, 256, 4 * 128):
        assert LIMIT + step - 1 < 1 << 31
        assert (LIMIT + step - 1) // step * step + step - 1 < 1 << 31
    assert LIMIT + 128 + 127 < 1 << 31
