"""Layer norm, rotary positions and tables, and the page pool without a GPU: the
references against torch's autograd and against differences, and every host
check of the entry points."""
import ctypes

import numpy as np
import pytest
import torch

from jagged_attention_recsys_gdpa_gb300 import _binding as B
from jagged_attention_recsys_gdpa_gb300 import build as build_mod
from tests import rows_ref as R

F = 1 << 20  # device pointers that no call below dereferences: each fails its checks first
INVALID, WORKSPACE, ALIGN = 1, 3, 4


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


# ------------------------------------------------------------------ references
@pytest.mark.parametrize("n", [1, 2, 3, 64])
@pytest.mark.parametrize("weights", [False, True])
def test_layer_norm_gradients_against_autograd_and_differences(n, weights):
    rng = np.random.default_rng(n)
    x, dy = rng.standard_normal((5, 2, n)) + 0.5, rng.standard_normal((5, 2, n))
    w, b = (rng.standard_normal(n), rng.standard_normal(n)) if weights else (None, None)
    eps = 1e-3
    y, mean, rstd = R.layer_norm(x, w, b, eps)
    t = torch.from_numpy(x).requires_grad_(True)
    tw, tb = (None, None) if w is None else (torch.from_numpy(v).requires_grad_(True) for v in (w, b))
    ty = torch.nn.functional.layer_norm(t, (n,), tw, tb, eps)
    assert np.allclose(y, ty.detach().numpy(), atol=1e-12)
    (ty * torch.from_numpy(dy)).sum().backward()
    dx, dw, db = R.layer_norm_grads(dy, x, w, rstd)
    assert np.allclose(dx, t.grad.numpy(), atol=1e-11)
    if weights:
        assert np.allclose(dw, tw.grad.numpy(), atol=1e-11) and np.allclose(db, tb.grad.numpy(), atol=1e-11)
    step = 1e-6
    for at in ((0, 0, 0), (4, 1, n - 1), (2, 0, n // 2)):
        up, down = x.copy(), x.copy()
        up[at] += step
        down[at] -= step
        diff = ((R.layer_norm(up, w, b, eps)[0] - R.layer_norm(down, w, b, eps)[0]) * dy).sum() / (2 * step)
        assert abs(diff - dx[at]) <= 1e-6 * (1 + abs(dx[at])) * max(1.0, rstd.max() ** 2)


def test_rotary_reference_is_a_complex_product_and_its_inverse_the_transpose():
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((6, 2, 10)).astype(np.float32))
    ang = rng.standard_normal((9, 4))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = np.array([0, 8, 3, -1, 9, 2])
    for layout in ("interleaved", "half"):
        y = R.rotary(x, cos, sin, pos, layout, False).numpy()
        f = x.numpy()
        a, b = (f[..., 0:8:2], f[..., 1:8:2]) if layout == "interleaved" else (f[..., :4], f[..., 4:8])
        ya, yb = (y[..., 0:8:2], y[..., 1:8:2]) if layout == "interleaved" else (y[..., :4], y[..., 4:8])
        for r in (0, 1, 2, 5):
            z = (a[r] + 1j * b[r]) * np.exp(1j * ang[pos[r]])
            assert np.allclose(ya[r], z.real, atol=1e-6) and np.allclose(yb[r], z.imag, atol=1e-6)
        assert np.all(y[3] == 0) and np.all(y[4] == f[4]) and np.all(y[[0, 1, 2, 5]][..., 8:] == f[[0, 1, 2, 5]][..., 8:])
        back = R.rotary(torch.from_numpy(y), cos, sin, pos, layout, True).numpy()
        assert np.allclose(back[[0, 1, 2, 4, 5]], f[[0, 1, 2, 4, 5]], atol=1e-6)


def test_pool_reference_restores_what_it_lends():
    pool = R.Pool(10, 4)
    table = np.full((3, 4), -1, np.int32)
    before = list(pool.free)
    slots = pool.assign(table, [0, 0, 0], [5, 0, 9], 14)
    assert slots[:6].tolist() == [0, 1, 2, 3, 4, 8] and table[2].tolist() == [2, 3, 4, -1]
    assert pool.assign(table, [5, 0, 9], [11, 16, 1], 28) is None
    assert pool.release(table, [5, 0, 9], None) and pool.free == before and np.all(table == -1)


# ------------------------------------------------------------------ host checks
def norm(lib, p=None, live=None, x=F, xr=256, xh=128, w=F * 2, b=F * 3, y=F * 4, yr=256, yh=128, mean=F * 5, rstd=F * 6,
         ws=None, ws_bytes=256, **kw):
    f = dict(rows=5, heads=2, N=128, type=1, weight_type=0, eps=1e-5, zero_behind=0)
    f.update(kw, x_strides=(xr, xh), y_strides=(yr, yh))
    return lib.jattn_layer_norm(ctypes.byref(B.Norm(**f)), live, x, w, b, y, mean, rstd, ws, ws_bytes, None)


def test_layer_norm_refusals(lib):
    assert norm(lib) == WORKSPACE  # all else is fine
    assert lib.jattn_layer_norm(None, None, F, F, F, F, F, F, F, 256, None) == INVALID
    for kw in (dict(rows=-1), dict(heads=0), dict(N=0), dict(N=16385), dict(rows=1 << 31, heads=1), dict(rows=1 << 30, heads=2),
               dict(type=3), dict(weight_type=2), dict(type=0, weight_type=1), dict(zero_behind=2), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(y=None), dict(w=None), dict(mean=None),
               dict(rstd=None), dict(xr=-1), dict(xh=-128), dict(xr=1 << 41),
               # rows of the output that share memory
               dict(yr=0), dict(yh=0), dict(yh=127), dict(yr=200), dict(yr=128, yh=256)):
        assert norm(lib, **kw) == INVALID, kw
    # heads behind all rows, a single head, and inputs whose rows are the same one
    for kw in (dict(yr=128, yh=640), dict(heads=1, yr=128, yh=0), dict(rows=1, yr=0), dict(xr=0, xh=0), dict(w=None, b=None),
               dict(b=None), dict(mean=None, rstd=None), dict(rows=0, x=None, y=None)):
        assert norm(lib, **kw) == WORKSPACE, kw
    for kw in (dict(x=F + 1), dict(y=4 * F + 1), dict(w=2 * F + 2), dict(b=3 * F + 2), dict(mean=5 * F + 2), dict(rstd=6 * F + 2),
               dict(live=F + 4), dict(type=0, x=F + 2)):
        assert norm(lib, **kw) == ALIGN, kw
    ok = dict(ws=F * 8)
    for kw in (dict(y=F + 2), dict(y=F, yr=512), dict(y=F + 1280 * 2 - 2), dict(w=4 * F), dict(b=4 * F + 2556), dict(mean=4 * F),
               dict(rstd=5 * F + 36), dict(mean=F), dict(rstd=2 * F), dict(live=4 * F), dict(live=5 * F + 32)):
        assert norm(lib, **ok, **kw) == INVALID, kw


def norm_bwd(lib, live=None, dy=F, dyr=256, dyh=128, x=2 * F, xr=256, xh=128, w=3 * F, mean=4 * F, rstd=5 * F, dx=6 * F, dxr=256,
             dxh=128, dw=7 * F, db=8 * F, scratch=9 * F, n=1 << 30, ws=None, **kw):
    f = dict(rows=5, heads=2, N=128, type=1, weight_type=0, eps=0.0, zero_behind=0)
    f.update(kw, x_strides=(xr, xh), y_strides=(dxr, dxh), dy_strides=(dyr, dyh))
    return lib.jattn_layer_norm_bwd(ctypes.byref(B.Norm(**f)), live, dy, x, w, mean, rstd, dx, dw, db, scratch, n, ws, 256, None)


def test_layer_norm_backward_refusals(lib):
    assert norm_bwd(lib) == WORKSPACE
    for kw in (dict(rows=-1), dict(N=0), dict(N=20000), dict(type=-1), dict(dy=None), dict(x=None), dict(dx=None), dict(mean=None),
               dict(rstd=None), dict(w=None), dict(dw=None), dict(dxr=0), dict(dxh=64), dict(dyr=-1), dict(xh=-1)):
        assert norm_bwd(lib, **kw) == INVALID, kw
    for kw in (dict(w=None, dw=None, db=None), dict(db=None), dict(dw=None, db=None, scratch=None), dict(dyr=0, dyh=0),
               dict(dx=F), dict(dx=2 * F)):
        assert norm_bwd(lib, **kw) == WORKSPACE, kw
    for kw in (dict(dy=F + 1), dict(x=2 * F + 1), dict(dx=6 * F + 1), dict(dw=7 * F + 2), dict(db=8 * F + 1), dict(mean=4 * F + 1),
               dict(rstd=5 * F + 2), dict(live=F + 4)):
        assert norm_bwd(lib, **kw) == ALIGN, kw


def rotary(lib, off=None, start=F, cos=2 * F, sin=3 * F, rows=100, x=4 * F, xr=256, xh=128, y=5 * F, yr=256, yh=128, ws=None, **kw):
    f = dict(B=6, total=6, heads=2, D=128, half=64, type=1, layout=0, inverse=0, zero_behind=0)
    f.update(kw, table_rows=rows, x_strides=(xr, xh), y_strides=(yr, yh))
    return lib.jattn_rotary(ctypes.byref(B.Rotary(**f)), off, start, cos, sin, x, y, ws, 256, None)


def test_rotary_refusals(lib):
    assert rotary(lib) == WORKSPACE
    for kw in (dict(total=-1), dict(total=1 << 31, B=1 << 31), dict(heads=0), dict(D=1, half=1), dict(D=16386), dict(half=0),
               dict(half=65), dict(type=9), dict(B=5), dict(off=F, B=0), dict(layout=2), dict(layout=-1), dict(inverse=2),
               dict(zero_behind=-1), dict(cos=None), dict(sin=None), dict(rows=0), dict(rows=1 << 31), dict(x=None), dict(y=None),
               dict(xr=-1), dict(yr=0), dict(yh=0), dict(heads=1 << 24)):
        assert rotary(lib, **kw) == INVALID, kw
    for kw in (dict(off=F, B=3), dict(start=None), dict(y=4 * F), dict(total=0, B=0, x=None, y=None), dict(xr=0, xh=0)):
        assert rotary(lib, **kw) == WORKSPACE, kw
    for kw in (dict(x=4 * F + 1), dict(y=5 * F + 1), dict(cos=2 * F + 2), dict(sin=3 * F + 1), dict(start=F + 4), dict(off=F + 2, B=3)):
        assert rotary(lib, **kw) == ALIGN, kw
    ok = dict(ws=8 * F)
    for kw in (dict(y=4 * F + 2), dict(y=4 * F, yr=512), dict(y=2 * F), dict(y=3 * F + 25598), dict(y=F), dict(off=5 * F + 8, B=3)):
        assert rotary(lib, **ok, **kw) == INVALID, kw


def tables(lib, cos=F, sin=2 * F, **kw):
    f = dict(first=0, rows=10, half=32, scaling=0, base=1e4, factor=1.0, original=4096.0, beta_fast=32.0, beta_slow=1.0)
    f.update(kw)
    return lib.jattn_rotary_tables(ctypes.byref(B.RotaryTables(**f)), cos, sin, None)


def test_rotary_tables_refusals(lib):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(first=-1), dict(rows=-1), dict(half=0), dict(half=513), dict(first=1 << 31, rows=1), dict(rows=(1 << 31) + 1),
               dict(first=1 << 62, rows=1 << 62), dict(base=1.0), dict(base=nan), dict(base=inf), dict(scaling=4), dict(scaling=-1),
               dict(scaling=1, factor=0.5), dict(scaling=2, factor=nan), dict(scaling=3, factor=inf), dict(scaling=2, half=1, factor=2.0),
               dict(scaling=3, original=0.0), dict(scaling=3, original=nan), dict(scaling=3, beta_slow=-1.0),
               dict(scaling=3, beta_fast=1.0), dict(scaling=3, beta_fast=inf), dict(cos=None), dict(sin=None), dict(sin=F),
               dict(sin=F + 1276)):
        assert tables(lib, **kw) == INVALID, kw
    for kw in (dict(cos=F + 2), dict(sin=2 * F + 1)):
        assert tables(lib, **kw) == ALIGN, kw


def assign(lib, pool=None, nb=3, total=7, off=F, start=2 * F, table=3 * F, max_pages=4, slots=4 * F, scratch=5 * F, n=1 << 20, ws=None,
           **kw):
    f = dict(n_pages=10, page_size=16, free_pages=6 * F, count=7 * F)
    f.update(kw)
    return lib.jattn_page_assign(ctypes.byref(B.PagePool(**f)), nb, total, off, start, table, max_pages, slots, scratch, n, ws, 256, None)


def release(lib, nb=3, lens=F, keep=2 * F, table=3 * F, max_pages=4, scratch=5 * F, n=1 << 20, ws=None, **kw):
    f = dict(n_pages=10, page_size=16, free_pages=6 * F, count=7 * F)
    f.update(kw)
    return lib.jattn_page_release(ctypes.byref(B.PagePool(**f)), nb, lens, keep, table, max_pages, scratch, n, ws, 256, None)


def test_page_pool_refusals(lib):
    size = ctypes.c_size_t(0)
    for total in (-1, 7):  # small calls need none
        assert lib.jattn_page_scratch_size(5, total, 4, ctypes.byref(size)) == 0 and size.value == 0
        assert lib.jattn_page_scratch_size(5000, total, 4, ctypes.byref(size)) == 0 and size.value >= 8 * 5000
    for args in ((0, 1, 1), (1 << 31, 1, 1), (1, -2, 1), (1, 1 << 31, 1), (1, 1, 0)):
        assert lib.jattn_page_scratch_size(*args, ctypes.byref(size)) == INVALID, args
    assert lib.jattn_page_scratch_size(5, 1, 1, None) == INVALID
    both = (dict(n_pages=0), dict(n_pages=1 << 31), dict(page_size=0), dict(page_size=24), dict(page_size=8192), dict(free_pages=None),
            dict(count=None), dict(nb=0), dict(table=None), dict(max_pages=0), dict(max_pages=1 << 28))
    for call in (assign, release):
        assert call(lib) == WORKSPACE
        for kw in both:
            assert call(lib, **kw) == INVALID, kw
        for kw in (dict(free_pages=6 * F + 2), dict(count=7 * F + 4), dict(table=3 * F + 2)):
            assert call(lib, **kw) == ALIGN, kw
        ok = dict(ws=10 * F)
        large = dict(nb=5000, table=11 * F, slots=12 * F) if call is assign else dict(nb=5000, table=11 * F)
        for kw in (dict(scratch=None), dict(scratch=5 * F + 8), dict(n=8)):
            assert call(lib, **ok, **large, **kw) == WORKSPACE, kw
        for kw in (dict(count=6 * F + 32), dict(table=6 * F + 36), dict(count=3 * F + 40)):
            assert call(lib, **ok, **kw) == INVALID, kw
        for kw in (dict(scratch=6 * F), dict(table=5 * F), dict(scratch=F)):
            assert call(lib, **dict(dict(ok, **large), **kw)) == INVALID, kw
    for kw in (dict(start=None), dict(total=-1), dict(total=1 << 31), dict(off=None)):
        assert assign(lib, **kw) == INVALID, kw
    for kw in (dict(off=None, total=3), dict(slots=None), dict(total=0)):
        assert assign(lib, **kw) == WORKSPACE, kw
    for kw in (dict(off=F + 4), dict(start=2 * F + 4), dict(slots=4 * F + 4)):
        assert assign(lib, **kw) == ALIGN, kw
    for kw in (dict(slots=F + 24), dict(slots=2 * F - 48), dict(slots=3 * F), dict(slots=6 * F), dict(start=7 * F), dict(off=3 * F)):
        assert assign(lib, ws=8 * F, **kw) == INVALID, kw
    assert release(lib, lens=None) == INVALID and release(lib, keep=None) == WORKSPACE
    assert release(lib, lens=F + 4) == ALIGN and release(lib, keep=2 * F + 2) == ALIGN
    assert release(lib, ws=8 * F, keep=3 * F) == INVALID


def test_error_string_of_the_pool(lib):
    assert "pool" in B.error_string(12) and B.error_string(13) == "unknown error code"


def test_python_refuses_host_tensors(lib):
    import jagged_attention_recsys_gdpa_gb300 as J

    x = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):
        J.layer_norm(x)
    with pytest.raises(ValueError):
        J.rotary(x, (torch.zeros(4, 4), torch.zeros(4, 4)))
    with pytest.raises(ValueError):
        J.rotary_tables(4, 8, device="cpu")
    for kw in (dict(dim=7), dict(dim=0), dict(dim=1026), dict(rows=-1), dict(first=-1), dict(rows=1 << 32), dict(scaling="other"),
               dict(scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            J.rotary_tables(**dict(dict(rows=4, dim=8), **kw))
    with pytest.raises(ValueError):
        J.PagePool(torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int64), 16)
