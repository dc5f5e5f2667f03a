"""Row operators without a GPU: host checks beside those of test_rows, and rules that their sources keep."""
import ctypes

import pytest

from jagged_attention_recsys_gdpa_gb300 import _binding as B
from jagged_attention_recsys_gdpa_gb300 import build as build_mod
from tests import test_rows as T


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def test_zero_stats_is_a_truth_value(lib):
    for value, code in ((0, T.WORKSPACE), (1, T.WORKSPACE), (2, T.INVALID), (-1, T.INVALID)):
        assert T.norm(lib, zero_stats=value) == code
    assert ctypes.sizeof(B.Norm) == 8 + 6 * 4 + 6 * 8 + 8
