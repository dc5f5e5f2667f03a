"""Refusals of the paged-cache entry points that need no GPU: index pointers that
are not aligned to their elements, and buffers that overlap."""
import ctypes

import pytest

from jagged_attention_recsys_gdpa_gb300 import _binding as B
from jagged_attention_recsys_gdpa_gb300 import build as build_mod

F = 1 << 20  # device pointers that no call below dereferences: each fails its checks first
INVALID, WORKSPACE, ALIGN = 1, 3, 4


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def cache(v=8 * F):
    return B.Cache(10, 16, 2, 128, 0, F, v, None, None)  # k: 10 * 16 * 2 * 128 * 2 = 81,920 bytes


def append(lib, c=None, off=F, start=F, table=F, ws=F):
    return lib.jattn_cache_append(ctypes.byref(c or cache()), 2, 5, off, start, table, 4, F, F, None, None, 0, ws, 256, None)


def read(lib, off=F, start=F, table=F, k=F, v=4 * F, ws=F):
    return lib.jattn_cache_read(ctypes.byref(cache()), 2, 5, off, start, table, 4, k, v, ws, 256, None)


def decode(lib, q_off=F, lens=F, table=F, q=F, o=4 * F, lse=8 * F, ws=F, act=0):
    p = B.params(2, 2, 64, 4, 128, act, 0, 0, 0.0, 0)  # q and o: 2,048 bytes, lse: 32
    return lib.jattn_decode(ctypes.byref(p), ctypes.byref(cache()), q_off, lens, table, 4, q, o, lse, F, 1 << 40, ws, 256, None)


def test_index_pointers_are_aligned_to_their_elements(lib):
    for call, wide, narrow in ((append, ("off", "start"), ("table",)), (read, ("off", "start"), ("table",)),
                               (decode, ("q_off", "lens"), ("table", "lse"))):
        for name in wide:
            for d in (1, 2, 4):
                assert call(lib, **{name: F + d, "ws": None}) == ALIGN, (name, d)
        for name in narrow:
            for d in (1, 2, 3):
                assert call(lib, **{name: F + d, "ws": None}) == ALIGN, (name, d)
            assert call(lib, **{name: F + 4, "ws": None}) == WORKSPACE  # fine so far
        assert call(lib, ws=None) == WORKSPACE


def test_buffers_that_overlap(lib):
    assert append(lib, cache(v=F)) == INVALID
    assert append(lib, cache(v=F + 81_920 - 16)) == INVALID
    for v in (F, F + 16, F - 16, F + 5 * 2 * 128 * 2 - 16):
        assert read(lib, v=v) == INVALID, v
    for o in (F, F + 16, F - 16, F + 2048 - 16, F - 2048 + 16):
        assert decode(lib, o=o) == INVALID, o
    for lse in (F, F - 28, F + 2044, 4 * F, 4 * F - 28, 4 * F + 2044):
        assert decode(lib, lse=lse) == INVALID, lse
