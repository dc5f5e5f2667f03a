"""The paged-cache entry points' host-side checks (no GPU), and the reference's
quantisation against its own definition."""
import ctypes

import numpy as np
import pytest
import torch

from jagged_attention_recsys_gdpa_gb300 import _binding as B
from jagged_attention_recsys_gdpa_gb300 import build as build_mod
from tests import paged_ref as R

F = 1 << 20  # a device pointer that no call below dereferences: each fails its checks first


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def make_cache(**kw):
    base = dict(n_pages=10, page_size=16, H=2, D=128, format=0, k=F, v=F, k_scales=None, v_scales=None)
    base.update(kw)
    return B.Cache(*[base[f[0]] for f in B.Cache._fields_])


BAD_CACHES = [(dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1), (dict(page_size=4), 1), (dict(page_size=24), 1),
              (dict(page_size=8192), 1), (dict(H=0), 1), (dict(D=96), 1), (dict(format=2), 1), (dict(k=None), 1),
              (dict(v=None), 1), (dict(format=1), 1), (dict(format=1, k_scales=F), 1), (dict(k_scales=F), 1),
              (dict(k_scales=F, v_scales=F), 1), (dict(k=F + 8), 4), (dict(v=F + 2), 4),
              (dict(format=1, k_scales=F + 2, v_scales=F), 4)]


def append(lib, c=None, B_=2, total=2, off=None, start=F, table=F, pages=4, k=F, v=F, cos=None, sin=None, rows=0, ws=F,
           ws_bytes=256):
    return lib.jattn_cache_append(ctypes.byref(c or make_cache()), B_, total, off, start, table, pages, k, v, cos, sin,
                                  rows, ws, ws_bytes, None)


def test_append_checks(lib):
    for kw, want in BAD_CACHES:
        assert append(lib, make_cache(**kw)) == want, kw
    for kw, want in [(dict(B_=0), 1), (dict(B_=1 << 31), 1), (dict(total=-1), 1), (dict(total=3), 1),
                     (dict(total=1 << 31, off=F), 1), (dict(start=None), 1), (dict(table=None), 1), (dict(pages=0), 1),
                     (dict(pages=1 << 27), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k=F + 8), 4),
                     (dict(cos=F), 1), (dict(sin=F, rows=5), 1), (dict(cos=F, sin=F, rows=0), 1),
                     (dict(cos=F + 4, sin=F, rows=5), 4), (dict(ws=None), 3), (dict(ws=F + 16), 3),
                     (dict(ws_bytes=128), 3)]:
        assert append(lib, **kw) == want, kw


def test_read_checks(lib):
    def read(c=None, B_=2, total=5, off=F, table=F, pages=4, k=F, v=F, ws=F, ws_bytes=256):
        return lib.jattn_cache_read(ctypes.byref(c or make_cache()), B_, total, off, None, table, pages, k, v, ws,
                                    ws_bytes, None)

    for kw, want in BAD_CACHES:
        assert read(make_cache(**kw)) == want, kw
    for kw, want in [(dict(B_=0), 1), (dict(total=-1), 1), (dict(off=None), 1), (dict(table=None), 1),
                     (dict(pages=0), 1), (dict(k=None), 1), (dict(v=F + 4), 4), (dict(ws=None), 3), (dict(ws_bytes=8), 3)]:
        assert read(**kw) == want, kw


def test_decode_checks(lib):
    def params(**kw):
        base = dict(B=2, total_q=2, total_kv=64, H=4, D=128, act=0, mask=0, window=0, scale=0.0, norm_by_lkv=0)
        base.update(kw)
        return B.params(**base)

    def decode(c=None, p=None, q_off=None, lens=F, table=F, pages=4, q=F, o=F + 4096, lse=F, scratch=F, scratch_bytes=1 << 40,
               ws=F, ws_bytes=256):
        return lib.jattn_decode(ctypes.byref(p or params()), ctypes.byref(c or make_cache()), q_off, lens, table, pages, q,
                                o, lse, scratch, scratch_bytes, ws, ws_bytes, None)

    for kw, want in BAD_CACHES:
        assert decode(make_cache(**kw)) == want, kw
    for kw, want in [(dict(p=params(H=3)), 1), (dict(p=params(D=64)), 1), (dict(p=params(total_kv=65)), 1),
                     (dict(p=params(total_q=3)), 1), (dict(p=params(act=7)), 1), (dict(p=params(mask=2)), 1),
                     (dict(p=params(norm_by_lkv=1)), 1), (dict(lens=None), 1), (dict(table=None), 1), (dict(pages=0), 1),
                     (dict(q=None), 1), (dict(o=None), 1), (dict(o=F), 1), (dict(lse=None), 1), (dict(q=F + 8), 4), (dict(o=F + 2), 4),
                     (dict(scratch=None), 3), (dict(scratch=F + 16), 3), (dict(scratch_bytes=0), 3), (dict(ws=None), 3),
                     (dict(ws=F + 8), 3), (dict(ws_bytes=64), 3)]:
        assert decode(**kw) == want, kw
    n = B.decode_scratch_size(ctypes.byref(params()), ctypes.byref(make_cache()))
    assert n > 0 and n % 256 == 0
    with pytest.raises(B.JattnError):
        B.decode_scratch_size(ctypes.byref(params(H=5)), ctypes.byref(make_cache()))


def test_error_names(lib):
    assert "page" in B.error_string(10) and "length" in B.error_string(11)


def test_reference_codes_match_the_type():
    """The reference's E4M3 grid and rounding are torch's float8_e4m3fn."""
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 2.0**e for e in range(-11, 9)])
    x = np.concatenate([x, R.E4M3, (R.E4M3[1:] + R.E4M3[:-1]) / 2, [0.0, -0.0, 464.0, 1e9]])
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_codes(x.astype(np.float32).astype(np.float64)), want)
    codes, e = R.quantise(np.array([[1.75] + [0.0] * 31, [3e38] * 32, [1e-45] * 32, [0.0] * 32]))
    assert e.ravel().tolist() == [119, 246, 0, 0]
    assert R.dequantise(codes, e)[0, 0] == 1.75
