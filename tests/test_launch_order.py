"""Kernels that are set up while the grid before them ends: each waits before it touches anything.

What an earlier grid wrote is promised to a thread that has waited for it, and to no other; so before the wait a
kernel that launch_after launches touches its shared memory at most, on every path (read here from the sources: a
kernel that reads too early gives the right answer nearly always).
"""
import os
import re

import pytest

from conftest import REPO

CSRC = os.path.join(REPO, "dense_gemm_epilogues_tcgen05_gb300", "csrc")


def kernels():
    """(file, kernel, text from its body's brace on) of the files that launch with launch_after."""
    for f in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        if not f.endswith(".cu") or "launch_after(" not in text:
            continue
        for m in re.finditer(r"__global__ void (?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\([^)]*\)\s*\{", text):
            yield f, m.group(1), text[m.end():]


def test_kernels_are_found():
    assert {k for _, k, _ in kernels()} >= {"route_kernel", "route_grad_kernel", "route_count_kernel", "route_rows_kernel",
                                            "rows_gather_kernel", "rows_combine_kernel", "rows_combine_grad_kernel",
                                            "mx_quantize_kernel", "mx_dequantize_kernel"}


SIZES = {"E", "P", "chunk", "top"}  # arguments that are no arrays


@pytest.mark.parametrize("file,kernel,body", [pytest.param(*k, id=k[1]) for k in kernels()])
def test_the_wait_comes_first(file, kernel, body):
    before = body[:body.index("begin_after();")]
    assert set(re.findall(r"\ba\.(\w+)", before)) <= SIZES, f"{file}: {kernel} uses an array before it waits"
    assert not re.search(r"\b(if|return|__ld|ld_|atomic|asm)\b|\ba\b(?!\.)", re.sub(r"if \(threadIdx\.x == 0\) \w+\[0\] = 0;", "", before)), \
        f"{file}: {kernel} does more than set up shared memory before it waits"
    assert before.count("{") == before.count("}"), f"{file}: {kernel} waits on some paths only"
    assert body.count("begin_after();", 0, body.find("__global__")) == 1


def test_the_wait_is_for_everything_before():
    text = open(os.path.join(CSRC, "launch.cuh")).read()
    body = text[text.index("begin_after() {"):]
    assert re.match(r"begin_after\(\) \{\s*grid_dep_wait\(\);\s*grid_dep_launch\(\);\s*\}", body)
