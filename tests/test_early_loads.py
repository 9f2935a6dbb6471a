"""A kernel that starts before its predecessor on the stream has ended reads nothing of it through the read-only intrinsic: the compiler
may move such a load ahead of the wait (it is no access that the wait's clobber of memory orders), and what the predecessor writes is not
constant for as long as the kernel runs.  Read from the sources, without a GPU: no run shows a load that happened to stay behind."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_router_gb300", "csrc")


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def _early():
    """Sources with a kernel that waits for its predecessor, and the headers that they take their loads from."""
    names = {os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))}
    early = {n for n in names if re.search(r"\bpdl_wait\(\)\s*;", _code(os.path.join(CSRC, n)))}
    for n in sorted(early):
        early |= set(re.findall(r'#include "([^"]+\.cuh)"', _code(os.path.join(CSRC, n)))) & names
    return sorted(early)


def test_finds_the_kernels():
    assert {"adapters.cu", "block_norm.cu", "linear.cu", "norm.cu", "rows.cuh"} <= set(_early())


@pytest.mark.parametrize("name", _early())
def test_no_read_only_intrinsic(name):
    found = [line.strip() for line in _code(os.path.join(CSRC, name)).splitlines() if re.search(r"\b__ldg\s*\(", line)]
    assert not found, found


def test_products_read_rows_by_ordered_loads():
    """Nor do the low-rank products by the non-coherent loads: their rows of x are a predecessor's results."""
    assert not re.search(r"\bldg_\w+\s*\(|ld\.global\.nc", _code(os.path.join(CSRC, "adapters.cu")))
