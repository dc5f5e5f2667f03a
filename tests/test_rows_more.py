"""Row operators without a GPU: host checks beside those of test_rows, and rules that their sources keep."""
import ctypes
import re

import pytest

from jagged_attention_recsys_gdpa_gb300 import _binding as B
from jagged_attention_recsys_gdpa_gb300 import build as build_mod
from tests import test_rows as T
from tests.test_paged_sources import code


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def test_zero_stats_is_a_truth_value(lib):
    for value, code in ((0, T.WORKSPACE), (1, T.WORKSPACE), (2, T.INVALID), (-1, T.INVALID)):
        assert T.norm(lib, zero_stats=value) == code
    assert ctypes.sizeof(B.Norm) == 8 + 6 * 4 + 6 * 8 + 8


@pytest.mark.parametrize("name", ["norm.cu", "norm_bwd.cu", "norm.cuh", "rotary.cu", "rows.cuh", "pages.cu", "pages.cuh"])
def test_no_read_only_loads_behind_a_programmatic_launch(name):
    """The rule of the paged cache's kernels: resident before the kernel that writes their inputs has ended, these read nothing
    through the read-only path either."""
    found = re.findall(r"__ldg|__ldc[asgv]|__ldlu|ld\.global\.nc|__restrict__", code(name))
    assert not found, found
    for text in re.findall(r"asm[^;]*\"ld\.global[^;]*;", code(name)):
        assert text.startswith("asm volatile"), text


@pytest.mark.parametrize("name,kernels", [("norm.cu", 1), ("norm_bwd.cu", 2), ("rotary.cu", 2), ("pages.cu", 6)])
def test_every_kernel_waits_for_the_one_before(name, kernels):
    """All are launched early: each waits (begin() of the pages' does) before it reads memory that another kernel writes."""
    bodies = re.split(r"__global__", code(name))[1:]
    assert len(bodies) == kernels
    for body in bodies:
        assert re.search(r"wait_for_dependency\(\)|\bbegin\(\)", body[:body.index("\n}\n")]), body[:120]
