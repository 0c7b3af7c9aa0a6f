"""The build's check of the kernels that trade registers, on reports as ptxas writes them."""
import os

import pytest

ENTRY = ("ptxas info    : Compiling entry function '_ZN5gb30012i8_tc_kernelILi{i}EEEv' for 'sm_103a'\n"
         "ptxas info    : Function properties for _ZN5gb30012i8_tc_kernelILi{i}EEEv\n"
         "    32 bytes stack frame, 68 bytes spill stores, 128 bytes spill loads\n"
         "ptxas info    : Used {r} registers, used 1 barriers, 32 bytes cumulative stack size\n")
OTHER = ("ptxas info    : Compiling entry function '_ZN5gb30013another_kernelEv' for 'sm_103a'\n"
         "ptxas info    : Used 80 registers, used 1 barriers\n")


@pytest.fixture(scope="module")
def bm():
    import __graft_entry__
    __graft_entry__.build()
    return __graft_entry__.build_module()


def test_accepts_the_written_count(bm):
    bm.check_registers(OTHER + ENTRY.format(i=0, r=72) + ENTRY.format(i=1, r=72) + OTHER)


@pytest.mark.parametrize("report", [ENTRY.format(i=0, r=72) + ENTRY.format(i=1, r=80), ENTRY.format(i=2, r=64), OTHER,
                                    ""], ids=["one_higher", "lower", "missing", "empty"])
def test_refuses_others(bm, report):
    with pytest.raises(RuntimeError, match="i8_tc_kernel"):
        bm.check_registers(report)


def test_this_build(bm):
    path = os.path.join(bm.BUILD_DIR, "ptxas_report.txt")
    if not os.path.exists(path):
        pytest.skip("the library was built elsewhere")
    with open(path) as f:
        bm.check_registers(f.read())
