"""Rules that the sources of the paged-cache kernels keep (no GPU)."""
import os
import re

import pytest

from jagged_attention_recsys_gdpa_gb300 import build as build_mod

CSRC = os.path.join(build_mod.HERE, "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["decode.cu", "cache.cu", "cache.cuh"])
def test_no_read_only_loads_behind_a_programmatic_launch(name):
    """These kernels may be resident before the kernel that writes their inputs has ended: loads through the read-only
    path, and intrinsics that the compiler may move before the wait, are not for them."""
    found = re.findall(r"__ldg|__ldc[asgv]|__ldlu|ld\.global\.nc|__restrict__", code(name))
    assert not found, found
    for text in re.findall(r"asm[^;]*\"ld\.global[^;]*;", code(name)):
        assert text.startswith("asm volatile"), text
