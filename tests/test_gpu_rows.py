"""Layer norm, rotary positions and their tables on the GPU against the plain
64-bit references in rows_ref."""
import ctypes

import numpy as np
import pytest
import torch

from tests import rows_ref as R
from tests.rows_ref import np64

pytestmark = pytest.mark.gpu

OFFSETS, ROPE = 5, 9
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, FP16, FP32]


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def clear(J):
    J.device_status()
    J.device_status()


def within(got, want, bound):
    got = np64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], np.broadcast_to(bound, got.shape)[bad][:5])


def rand(shape, dtype, seed, shift=0.0, std=1.0):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * std + shift
    return x.to(dtype)


def strided(x, how):
    """x (CPU) on the GPU: dense, heads of a wider fused tensor, one element off every alignment, or heads first."""
    x = x.cuda()
    if how == "dense" or x.dim() == 2:
        return x
    n, h, d = x.shape
    if how == "fused":
        whole = torch.full((n, h + 3, d), float("nan"), dtype=x.dtype, device="cuda")
        view = whole[:, 1:1 + h]
    elif how == "odd":
        whole = torch.full((n * (h * d + 1) + 1,), float("nan"), dtype=x.dtype, device="cuda")
        view = whole[1:].view(n, h * d + 1)[:, :h * d].unflatten(1, (h, d))
    else:
        view = torch.empty((h, n, d), dtype=x.dtype, device="cuda").transpose(0, 1)
    view.copy_(x)
    return view


# ------------------------------------------------------------------ layer norm
SIZES = [1, 2, 3, 7, 8, 9, 31, 32, 33, 64, 96, 100, 127, 128, 129, 250, 256, 257, 512, 520, 1000, 1001, 1024, 1032, 2047, 2048, 2056,
         4096, 4104, 5000, 8192, 8193, 8200, 12345, 16383, 16384]


def check_norm(J, x, w, b, dy, eps=1e-5, off=None, live=None, depth=None):
    """Both directions of rows x (and dy) on the GPU against the references; live: rows that count."""
    live = x.shape[0] if live is None else live
    f64 = lambda t: None if t is None else np64(t)  # noqa: E731
    x64, w64, b64, dy64 = np64(x)[:live], f64(w), f64(b), np64(dy)[:live]
    y, mean, rstd = J.layer_norm_forward(x, w, b, eps=eps, off=off)
    assert y.dtype == x.dtype and y.is_contiguous() and mean.dtype == rstd.dtype == FP32
    want = R.layer_norm(x64, w64, b64, eps)
    eps32 = float(np.float32(eps))
    bound = R.layer_norm_bounds(x64, w64, b64, eps32, x.dtype)
    for got, v, e in zip((y, mean, rstd), want, bound):
        within(got[:live], v, e)
        assert bool((got[live:] == 0).all())
    dx, dw, db = J.layer_norm_backward(dy, x, w, mean, rstd, off=off)
    r64 = np64(rstd)[:live]
    want = R.layer_norm_grads(dy64, x64, w64, r64)
    # rows of a lane one after another, then a CTA's groups and the partial rows: no more additions than rows, or
    # 600 where there are more than the grid takes at a time
    rows = x64.size // x64.shape[-1]
    depth = (rows if depth is None else depth) + 64
    bound = R.layer_norm_grad_bounds(dy64, x64, w64, r64, x.dtype, FP32 if w is None else w.dtype, depth)
    within(dx[:live], want[0], bound[0])
    assert bool((dx[live:] == 0).all())
    if w is None:
        assert dw is None and db is None
    else:
        assert dw.dtype == db.dtype == w.dtype
        within(dw, want[1], bound[1])
        within(db, want[2], bound[2])
    assert J.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", SIZES)
def test_layer_norm_sizes(n, dtype):
    """Every shape of lanes and vectors, one size under and over each, from one row to more than a CTA's."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    for rows, wide in ((1, True), (37, False)):
        t = FP32 if wide else dtype
        check_norm(J, rand((rows, n), dtype, n, 0.7).cuda(), rand((n,), t, n + 1, 1.0).cuda(), rand((n,), t, n + 2).cuda(),
                   rand((rows, n), dtype, n + 3).cuda())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [249, 253, 381, 505, 509, 761, 763, 1009, 1010, 1019, 1533, 2041, 2045, 3001, 4087, 4091, 6129, 6133, 6137, 8177, 8185])
def test_layer_norm_rows_that_start_anywhere(n, dtype):
    """Odd widths around each shape's limits, of rows that share a shift in fewer and more than one turn of the grid."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    w, b = rand((n,), FP32, n + 1, 1.0).cuda(), rand((n,), FP32, n + 2).cuda()
    for rows in (1, 9, 70):
        check_norm(J, rand((rows, n), dtype, n, 0.7).cuda(), w, b, rand((rows, n), dtype, n + 3).cuda())
    # many rows: each as in a small call that starts at the same place
    x = rand((64, n), dtype, n).cuda()
    y, mean, rstd = J.layer_norm_forward(x, w, b)
    y2, mean2, rstd2 = J.layer_norm_forward(x.repeat(100, 1), w, b)
    assert torch.equal(y2, y.repeat(100, 1)) and torch.equal(mean2, mean.repeat(100)) and torch.equal(rstd2, rstd.repeat(100))
    assert J.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [101, 1001, 5001, 7001])
def test_layer_norm_in_padded_buffers(n, dtype):
    """Odd widths in buffers whose rows are whole vectors, with heads beside them, from an odd place on: what lies around the rows
    is NaN and stays as it is."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    wide = -(-(n + 3) // 8) * 8
    x, dy = (rand((41, 2, n), dtype, s, 0.3) for s in (1, 2))
    w, b = rand((n,), dtype, 3, 1.0).cuda(), rand((n,), dtype, 4).cuda()

    def inside(t, start):
        whole = torch.full((41, 3, wide), float("nan"), dtype=dtype, device="cuda")
        view = whole[:, :2, start:start + n]
        if t is not None:
            view.copy_(t)
        return whole, view

    for start in (0, 3):
        xs, ds = inside(x, start)[1], inside(dy, start)[1]
        whole, out = inside(None, start)
        y, mean, rstd = J.layer_norm_forward(xs, w, b, out=out)
        bounds = R.layer_norm_bounds(np64(x), np64(w), np64(b), float(np.float32(1e-5)), dtype)
        for got, v, e in zip((y, mean, rstd), R.layer_norm(np64(x), np64(w), np64(b), 1e-5), bounds):
            within(got, v, e)
        grads, gout = inside(None, start)
        got = J.layer_norm_backward(ds, xs, w, mean, rstd, out=gout)
        args = np64(dy), np64(x), np64(w), np64(rstd)
        for g, v, e in zip(got, R.layer_norm_grads(*args), R.layer_norm_grad_bounds(*args, dtype, dtype, 82 + 64)):
            within(g, v, e)
        for buffer in (whole, grads):
            buffer[:, :2, start:start + n] = float("nan")
            assert bool(torch.isnan(buffer).all())
    assert J.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("how", ["dense", "fused", "odd", "heads first"])
@pytest.mark.parametrize("n", [64, 128, 100, 1024])
def test_layer_norm_heads_and_strides(n, how, dtype):
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    x, dy = (rand((53, 5, n), dtype, s, 0.3) for s in (1, 2))
    w, b = rand((n,), dtype, 3, 1.0).cuda(), rand((n,), dtype, 4).cuda()
    check_norm(J, strided(x, how), w, b, strided(dy, "dense" if how == "odd" else how))
    check_norm(J, strided(x, how), None, None, strided(dy, how))
    # an output of the caller's, laid out the same, gets what a dense one does; a bias is not needed
    y, mean, rstd = J.layer_norm_forward(strided(x, how), w)
    to = strided(torch.zeros_like(x), how)
    y2, _, _ = J.layer_norm_forward(strided(x, how), w, out=to)
    assert y2 is to
    within(to, np64(y), 2 * R.layer_norm_bounds(np64(x), np64(w), None, 1e-5, dtype)[0])
    dx, dw, db = J.layer_norm_backward(strided(dy, how), strided(x, how), w, mean, rstd, bias=False)
    assert db is None
    assert J.device_status() == 0


def test_layer_norm_broadcast_rows():
    """Rows and gradients that are one row expanded (a gradient of a sum, a shared query)."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    w, b = rand((128,), FP32, 3, 1.0).cuda(), rand((128,), FP32, 4).cuda()
    x = rand((1, 1, 128), BF16, 5).cuda().expand(40, 3, 128)
    dy = rand((1, 3, 128), BF16, 6).cuda().expand(40, 3, 128)
    check_norm(J, x, w, b, dy)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [128, 130, 2000])
def test_layer_norm_rows_far_from_zero(n, dtype):
    """Means thousands of times the spread, constant rows, rows of zeros, tiny and large values."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    x = rand((12, n), torch.float64, n)
    x[0:3] += torch.tensor([3000.0, -500.0, 40000.0])[:, None]
    x[3] = 7.25
    x[4] = 0.0
    x[5] *= 1e-4
    x[6] *= 1000.0
    x[7] = 0.0
    x[7, n // 2] = 30000.0
    if dtype != FP16:
        x[8] *= 1e15
        x[9] *= 1e-18
    x = x.to(dtype)
    w, b, dy = rand((n,), FP32, 3, 1.0).cuda(), rand((n,), FP32, 4).cuda(), rand((12, n), dtype, 5)
    for eps in (1e-5, 1e-12, 1.0):
        if dtype == FP16 and eps < 1e-5:
            continue  # a gradient of a constant row would pass fp16's range
        check_norm(J, x.cuda(), w, b, dy.cuda(), eps=eps)


@pytest.mark.parametrize("n", [128, 100, 4096])
@pytest.mark.parametrize("heads", [1, 3])
def test_layer_norm_padded_batches(n, heads):
    """Rows behind off[-1] hold NaN: they reach nothing, and outputs of the caller's stay as they were there."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    for live, total in ((0, 5), (1, 9), (29, 40), (40, 40)):
        off = cu(np.array([0, live // 2, live]))
        x, dy = rand((total, heads, n), BF16, 1), rand((total, heads, n), BF16, 2)
        x[live:] = dy[live:] = float("nan")
        x, dy = x.cuda(), dy.cuda()
        w, b = rand((n,), FP32, 3, 1.0).cuda(), rand((n,), FP32, 4).cuda()
        check_norm(J, x, w, b, dy, off=off, live=live)
        out = torch.full_like(x, 5.0)
        y, mean, rstd = J.layer_norm_forward(x, w, b, off=off, out=out)
        assert bool((out[live:] == 5.0).all()) and bool(torch.isfinite(out[:live]).all())
        out = torch.full_like(x, 5.0)
        J.layer_norm_backward(dy, x, w, mean, rstd, off=off, out=out)
        assert bool((out[live:] == 5.0).all()) and bool(torch.isfinite(out[:live]).all())
    for bad, rows in ((-1, 0), (41, 40), (2**40, 40), (-2**62, 0)):
        y, _, _ = J.layer_norm_forward(x, w, b, off=cu(np.array([0, bad])))
        assert J.device_status() == OFFSETS
        whole, _, _ = J.layer_norm_forward(x, w, b)
        assert torch.equal(y[:rows], whole[:rows]) and bool((y[rows:] == 0).all())
    assert J.device_status() == 0


def test_layer_norm_without_rows():
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    w = torch.ones(64, device="cuda")
    x = torch.zeros(0, 3, 64, dtype=BF16, device="cuda")
    y, mean, rstd = J.layer_norm_forward(x, w, w)
    assert y.shape == x.shape and mean.shape == (0, 3)
    dx, dw, db = J.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == x.shape and bool((dw == 0).all()) and bool((db == 0).all())
    assert J.device_status() == 0


@pytest.mark.parametrize("n", [128, 100, 2048])
def test_layer_norm_in_place(n):
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    x, dy, w = rand((41, 2, n), BF16, 1).cuda(), rand((41, 2, n), BF16, 2).cuda(), rand((n,), FP32, 3, 1.0).cuda()
    y, mean, rstd = J.layer_norm_forward(x, w)
    z = x.clone()
    assert J.layer_norm_forward(z, w, out=z)[0] is z and torch.equal(z, y)
    dx, dw, db = J.layer_norm_backward(dy, x, w, mean, rstd)
    for which in (0, 1):
        pair = [dy.clone(), x.clone()]
        got = J.layer_norm_backward(pair[0], pair[1], w, mean, rstd, out=pair[which])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    for shift in (1, n):
        flat = torch.zeros(82 * n + shift, dtype=BF16, device="cuda")
        with pytest.raises(J.JattnError):
            J.layer_norm_forward(flat[:82 * n].view(41, 2, n), w, out=flat[shift:].view(41, 2, n))
    with pytest.raises(J.JattnError):
        J.layer_norm_forward(x, w, out=x[:1].expand(41, 2, n))
    # the heads of one fused tensor into others of it: their spans meet
    fused = torch.zeros(41, 4, n, dtype=BF16, device="cuda")
    with pytest.raises(J.JattnError):
        J.layer_norm_forward(fused[:, :2], w, out=fused[:, 2:])
    assert J.device_status() == 0


@pytest.mark.parametrize("n", [64, 1000, 1024])
def test_layer_norm_infinities_stay_in_their_row(n):
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    x, dy, w = rand((50, n), BF16, 1).cuda(), rand((50, n), BF16, 2).cuda(), rand((n,), FP32, 3, 1.0).cuda()
    y, mean, rstd = J.layer_norm_forward(x, w)
    dx, _, _ = J.layer_norm_backward(dy, x, w, mean, rstd)
    others = torch.arange(50) != 17
    for value in (float("inf"), float("-inf"), float("nan")):
        z = x.clone()
        z[17, n // 3] = value
        y2, m2, r2 = J.layer_norm_forward(z, w)
        assert not bool(torch.isfinite(y2[17]).any())
        assert torch.equal(y2[others], y[others]) and torch.equal(m2[others], mean[others]) and torch.equal(r2[others], rstd[others])
        dx2, _, _ = J.layer_norm_backward(dy, z, w, m2, r2)
        assert torch.equal(dx2[others], dx[others]) and not bool(torch.isfinite(dx2[17]).any())
    assert J.device_status() == 0


@pytest.mark.parametrize("rows,n,dtype", [(200_003, 128, BF16), (100_001, 64, FP16), (20_011, 1001, BF16), (9_001, 2048, FP32)])
def test_layer_norm_many_rows(rows, n, dtype):
    """More rows than the grid takes at a time: against the same rows in small calls, bit for bit (rows that start at another place
    within 16 bytes are summed in another order: both are within the bounds of rows_ref), and the weight's gradient against the
    64-bit sum. Lanes add at most 600 rows here, a CTA's groups 64, the join 128."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = (torch.randn(rows, n, generator=g, device="cuda").add_(0.5).to(dtype) for _ in range(2))
    w, b = rand((n,), FP32, 3, 1.0).cuda(), rand((n,), FP32, 4).cuda()
    y, mean, rstd = J.layer_norm_forward(x, w, b)
    dx, dw, db = J.layer_norm_backward(dy, x, w, mean, rstd)
    for first in (0, 12_345 % rows, rows - 100):
        part = slice(first, first + 100)
        y2, m2, r2 = J.layer_norm_forward(x[part], w, b)
        d2 = J.layer_norm_backward(dy[part], x[part], w, mean[part], rstd[part])[0]
        if first * n * x.element_size() % 16 == 0:
            assert torch.equal(y2, y[part]) and torch.equal(m2, mean[part]) and torch.equal(r2, rstd[part])
            assert torch.equal(d2, dx[part])
        else:
            x64, w64 = np64(x[part]), np64(w)
            bounds = R.layer_norm_bounds(x64, w64, np64(b), float(np.float32(1e-5)), dtype)
            for got, of, bound in zip((y2, m2, r2), (y, mean, rstd), bounds):
                within(got, np64(of[part]), 2 * bound)
            bound = R.layer_norm_grad_bounds(np64(dy[part]), x64, w64, np64(rstd[part]), dtype, FP32, 164)[0]
            within(d2, np64(dx[part]), 2 * bound)
    xd, dyd, r = x.double(), dy.double(), rstd.double()[:, None]
    m = xd.mean(-1, keepdim=True)
    h = (xd - m) * r
    # as in rows_ref: h is off by at most 100 u (1 + |h|) here (|m| rstd is about 0.5, mean|x - m| rstd below 1), the sums by 800 u
    size = (dyd.abs() * (1 + h.abs())).sum(0)
    assert bool(((dw.double() - (dyd * h).sum(0)).abs() <= 900 * R.U * size).all())
    assert bool(((db.double() - dyd.sum(0)).abs() <= 900 * R.U * dyd.abs().sum(0)).all())
    again = J.layer_norm_backward(dy, x, w, mean, rstd)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)
    assert J.device_status() == 0


def test_layer_norm_beyond_32_bit_offsets():
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    n, rows = 4096, (1 << 32) // 4096 + 300
    if torch.cuda.mem_get_info()[0] < 6 * rows * n * 2:
        pytest.skip("not enough free memory")
    x = torch.zeros(rows, n, dtype=BF16, device="cuda")
    far = rand((300, n), BF16, 7).cuda()
    x[-300:] = far
    w = rand((n,), FP32, 3, 1.0).cuda()
    y, mean, rstd = J.layer_norm_forward(x, w)
    y2, m2, r2 = J.layer_norm_forward(far, w)
    assert torch.equal(y[-300:], y2) and torch.equal(mean[-300:], m2) and torch.equal(rstd[-300:], r2)
    dx, dw, db = J.layer_norm_backward(x, x, w, mean, rstd)
    dx2, _, _ = J.layer_norm_backward(far, far, w, m2, r2)
    assert torch.equal(dx[-300:], dx2)
    assert J.device_status() == 0


def test_layer_norm_autograd():
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    for dtype, wt in ((BF16, FP32), (FP32, FP32), (FP16, FP16)):
        base = rand((33, 4, 128), dtype, 1, 0.3).cuda()
        w0, b0, dy = rand((128,), wt, 2, 1.0).cuda(), rand((128,), wt, 3).cuda(), rand((33, 4, 128), dtype, 4).cuda()
        _, mean, rstd = J.layer_norm_forward(base, w0, b0)
        want = J.layer_norm_backward(dy, base, w0, mean, rstd)
        x, w, b = (t.clone().requires_grad_(True) for t in (base, w0, b0))
        J.layer_norm(x, w, b).backward(dy)
        for leaf, g in zip((x, w, b), want):
            assert torch.equal(leaf.grad, g)
        x.grad = None
        J.layer_norm(x).backward(dy)  # without a weight
        assert torch.equal(x.grad, J.layer_norm_backward(dy, base, None, mean, rstd)[0])
        w.grad = b.grad = None
        J.layer_norm(base, w, b).sum().backward()  # an expanded gradient, and no leaf x
        ones = J.layer_norm_backward(torch.ones_like(base), base, w0, mean, rstd)
        assert torch.equal(w.grad, ones[1]) and torch.equal(b.grad, ones[2])
        frozen = J.layer_norm(x, w0, b0)
        frozen.backward(dy)
    assert J.device_status() == 0


def test_layer_norm_gradient_against_differences():
    """All gradients of L = sum(dy y) against central differences of the 64-bit forward (step 1e-5: their error is below 1e-8
    here, as third derivatives stay below 100 and L below 1,000)."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    x, dy, w, b = rand((6, 40), FP32, 1), rand((6, 40), FP32, 2), rand((40,), FP32, 4, 1.0), rand((40,), FP32, 5)
    _, mean, rstd = J.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    got = J.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    x64, dy64, w64, b64 = (np64(t) for t in (x, dy, w, b))
    # the reference takes the kernel's rstd, off by 30 u: as a share of a gradient no more than 100 u
    bounds = R.layer_norm_grad_bounds(dy64, x64, w64, R.layer_norm(x64, w64, b64, 1e-5)[2], FP32, FP32, 70)
    for which, (grad, bound) in enumerate(zip(got, bounds)):
        args = [x64, w64, b64]
        diff = np.zeros_like(args[which])
        for at in np.ndindex(diff.shape):
            up, down = list(args), list(args)
            up[which], down[which] = args[which].copy(), args[which].copy()
            up[which][at] += 1e-5
            down[which][at] -= 1e-5
            diff[at] = ((R.layer_norm(*up, 1e-5)[0] - R.layer_norm(*down, 1e-5)[0]) * dy64).sum() / 2e-5
        within(grad, diff, bound + 100 * R.U * (np.abs(diff) + 20) + 1e-8)
    assert J.device_status() == 0


def test_layer_norm_on_streams_and_in_graphs():
    """Calls at the same time on several streams, and two captured training steps replayed at the same time on new rows."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    x, dy, w = rand((3001, 2, 128), BF16, 1).cuda(), rand((3001, 2, 128), BF16, 2).cuda(), rand((128,), FP32, 3, 1.0).cuda()
    y, mean, rstd = J.layer_norm_forward(x, w, w)
    want = J.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(24):
        with torch.cuda.stream(streams[i % 3]):
            got.append((J.layer_norm_forward(x, w, w)[0], *J.layer_norm_backward(dy, x, w, mean, rstd)))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], y) and all(torch.equal(a, b) for a, b in zip(g[1:], want))
    sides = []
    for i in range(2):
        xs, ds = torch.zeros_like(x), torch.zeros_like(dy)
        graph, res = torch.cuda.CUDAGraph(), []
        with torch.cuda.graph(graph):
            yy, m, r = J.layer_norm_forward(xs, w, w)
            res += [yy, *J.layer_norm_backward(ds, xs, w, m, r)]
        sides.append((xs, ds, graph, res, streams[i]))
    torch.cuda.synchronize()
    for t in range(20):
        for i, (xs, ds, graph, res, st) in enumerate(sides):
            with torch.cuda.stream(st):
                xs.copy_(x.roll(t + i, 0))
                ds.copy_(dy.roll(t + i, 0))
                graph.replay()
    torch.cuda.synchronize()
    for i, (xs, ds, graph, res, st) in enumerate(sides):
        yy, m, r = J.layer_norm_forward(xs, w, w)
        for a, b in zip(res, (yy, *J.layer_norm_backward(ds, xs, w, m, r))):
            assert torch.equal(a, b)
    assert J.device_status() == 0


def test_in_place_calls_count_as_writes():
    """Autograd refuses a backward pass through rows that a call has overwritten since."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    tables = J.rotary_tables(8, 16)
    for write in (lambda x: J.layer_norm_forward(x, out=x), lambda x: J.rotary(x, tables, out=x),
                  lambda x: J.layer_norm_backward(torch.ones_like(x), x, None, x[..., 0].contiguous(), x[..., 0].contiguous(), out=x)):
        x = rand((8, 2, 16), FP32, 1).cuda()
        w = torch.ones(16, device="cuda", requires_grad=True)
        loss = (x * w).sum()  # keeps x for w's gradient
        write(x)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
        with torch.inference_mode():
            z = torch.ones(8, 2, 16, device="cuda")
            write(z)
        write(z)
    assert J.device_status() == 0


def test_layer_norm_python_refusals():
    import jagged_attention_recsys_gdpa_gb300 as J

    x = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    J.layer_norm_forward(x, w, w)
    off = torch.tensor([0, 4], device="cuda")
    for kw in (dict(x=x.double()), dict(x=x[0, 0]), dict(x=x.transpose(1, 2)), dict(x=x[None]), dict(w=w[:5]), dict(w=w.double()),
               dict(w=w.half()), dict(w=w.cpu()), dict(b=w.bfloat16()), dict(w=None), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(off=off.int()), dict(off=off.cpu()), dict(off=off[:0]), dict(out=x.float()), dict(out=x[:2]),
               dict(out=x.clone().requires_grad_(True)), dict(x=x[:, :0]), dict(x=x[..., :0], w=w[:0], b=w[:0]),
               dict(x=torch.zeros(2, 16385, device="cuda"), w=None, b=None)):
        kw = dict(dict(x=x, w=w, b=w), **kw)
        with pytest.raises(ValueError):
            J.layer_norm_forward(kw.pop("x"), kw.pop("w"), kw.pop("b"), **kw)
    m = torch.zeros(4, 2, device="cuda")
    J.layer_norm_backward(x, x, w, m, m)
    for kw in (dict(dy=x.float()), dict(dy=x[:2]), dict(m=m.half()), dict(m=m[:, :1]), dict(r=m.t()), dict(r=m.cpu()), dict(w=w[:3]),
               dict(out=x.float())):
        kw = dict(dict(dy=x, w=w, m=m, r=m), **kw)
        with pytest.raises(ValueError):
            J.layer_norm_backward(kw.pop("dy"), x, kw.pop("w"), kw.pop("m"), kw.pop("r"), **kw)
    assert J.device_status() == 0


# ------------------------------------------------------------------ rotary positions
def angles(rows, half, seed=0):
    a = np.random.default_rng(seed).uniform(-4, 4, (rows, half))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def same(got, want):
    assert got.shape == want.shape and got.dtype == want.dtype
    got = got.cpu()
    bits = {2: torch.int16, 4: torch.int32}[got.element_size()]
    # a product's zero may have either sign where a value is zero
    equal = (got.contiguous().view(bits) == want.contiguous().view(bits)) | ((got == 0) & (want == 0))
    assert bool(equal.all()), torch.argwhere(~equal)[:5]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,half", [(2, 1), (3, 1), (64, 32), (64, 16), (96, 48), (128, 64), (128, 8), (80, 12), (100, 50), (33, 16),
                                    (256, 128), (2000, 1000), (40, 4)])
def test_rotary_layouts(D, half, dtype, layout):
    """Bit for bit the formula's values, whole and part heads, vectors and single values, one and several heads."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    cos, sin = angles(70, half)
    off = np.array([0, 5, 5, 6, 43])
    start = np.array([3, 0, 69, 20])
    for heads in (1, 3, 8):
        x = rand((47, heads, D), dtype, D + heads)
        pos = R.positions(47, off, start)
        for inverse in (False, True):
            y = J.rotary(x.cuda(), (cu(cos), cu(sin)), off=cu(off), start=cu(start), layout=layout, inverse=inverse)
            same(y, R.rotary(x, cos, sin, pos, layout, inverse))
    assert J.device_status() == 0


@pytest.mark.parametrize("how", ["dense", "fused", "odd", "heads first"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rotary_strides_and_in_place(layout, how):
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    cos, sin = angles(60, 32)
    t = (cu(cos), cu(sin))
    for dtype, heads, D in ((BF16, 5, 128), (FP32, 2, 64), (FP16, 4, 70)):
        x = rand((50, heads, D), dtype, 1)
        want = R.rotary(x, cos, sin, R.positions(50, None, None), layout, False)
        view = strided(x, how)
        same(J.rotary(view, t, layout=layout), want)
        to = strided(torch.zeros_like(x), how)
        assert J.rotary(view, t, layout=layout, out=to) is to
        same(to, want)
        whole = view.clone(memory_format=torch.contiguous_format)
        assert J.rotary(view, t, layout=layout, out=view) is view
        same(view, want)
        with pytest.raises(J.JattnError):
            J.rotary(whole, t, layout=layout, out=whole[:1].expand_as(whole))
    fused = torch.zeros(10, 4, 64, device="cuda")
    with pytest.raises(J.JattnError):
        J.rotary(fused[:, :2], t, layout=layout, out=fused[:, 1:3])
    assert J.device_status() == 0


@pytest.mark.parametrize("heads,D", [(1, 64), (8, 128), (3, 34)])
def test_rotary_positions(heads, D):
    """Positions by sequences and by rows, skipped ones, padding, and those behind the tables."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    cos, sin = angles(40, D // 2)
    t = (cu(cos), cu(sin))
    x = rand((30, heads, D), BF16, 1)
    off = np.array([0, 0, 7, 8, 8, 25])
    for start in (None, np.array([0, 4, 39, 100, 23]), np.array([-1, -5, 0, 0, -2**60])):
        pos = R.positions(30, off, start)
        y = J.rotary(x.cuda(), t, off=cu(off), start=None if start is None else cu(start))
        assert J.device_status() == 0
        same(y, R.rotary(x, cos, sin, pos, "interleaved", False))
        out = torch.full_like(x, 9.0).cuda()
        J.rotary(x.cuda(), t, off=cu(off), start=None if start is None else cu(start), out=out)
        keep = torch.from_numpy(pos < 0)
        assert bool((out.cpu()[keep] == 9.0).all())
        same(out.cpu()[~keep], R.rotary(x, cos, sin, pos, "interleaved", False)[~keep])
        z = x.cuda()
        J.rotary(z, t, off=cu(off), start=None if start is None else cu(start), out=z)
        same(z.cpu()[keep], x[keep])
    rows = np.random.default_rng(3).integers(-3, 40, 30)
    same(J.rotary(x.cuda(), t, start=cu(rows)), R.rotary(x, cos, sin, R.positions(30, None, rows), "interleaved", False))
    assert J.device_status() == 0
    for far in (40, 2**31, 2**40, 2**62, 2**63 - 1):
        rows[5] = far
        same(J.rotary(x.cuda(), t, start=cu(rows)), R.rotary(x, cos, sin, R.positions(30, None, rows), "interleaved", False))
        assert J.device_status() == ROPE
        start = np.array([0, far, 0, 0, 0])
        y = J.rotary(x.cuda(), t, off=cu(off), start=cu(start))
        assert J.device_status() == ROPE
        same(y[:7], x[:7])
    for bad in ([0, 9, 3, 8, 8, 25], [1, 1, 7, 8, 8, 25], [0, 0, 7, 8, 8, 31], [0, -4, 7, 8, 8, 25], [0, 2**60, 7, 8, 8, 25]):
        J.rotary(x.cuda(), t, off=cu(np.array(bad)))
        assert J.device_status() == OFFSETS, bad
    same(J.rotary(x.cuda(), t), R.rotary(x, cos, sin, np.arange(30), "interleaved", False))
    assert J.rotary(x.cuda()[:0], t).shape == (0, heads, D)
    assert J.device_status() == 0


def test_rotary_many_rows():
    """Calls of several heads and rows a thread, padded, with thousands of sequences: against the formula on the GPU."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    g = torch.Generator(device="cuda").manual_seed(5)
    for heads, D, half, B in ((8, 128, 64, 900), (10, 64, 16, 33), (3, 80, 40, 4000), (5, 50, 13, 7)):
        lens = torch.randint(0, 400_000 // (heads * B) + 2, (B,), generator=torch.Generator().manual_seed(B))
        off = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).cuda()
        n = int(off[-1])
        x = torch.randn(n + 11, heads, D, generator=g, device="cuda").to(BF16)
        start = torch.randint(0, 1000, (B,), generator=g, device="cuda")
        cos, sin = (torch.randn(int(lens.max()) + 1000, half, generator=g, device="cuda") for _ in range(2))
        y = J.rotary(x, (cos, sin), off=off, start=start, layout="half")
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), lens.cuda())
        pos = torch.arange(n, device="cuda") - off[b] + start[b]
        a, e = x[:n, :, :half].float(), x[:n, :, half:2 * half].float()
        c, s = cos[pos][:, None], sin[pos][:, None]
        assert torch.equal(y[:n, :, :half], (a * c - e * s).to(BF16)) and torch.equal(y[:n, :, half:2 * half], (a * s + e * c).to(BF16))
        assert torch.equal(y[:n, :, 2 * half:], x[:n, :, 2 * half:]) and bool((y[n:] == 0).all())
    assert J.device_status() == 0


def test_rotary_agrees_with_rope():
    """The interleaved layout is rope's: the same numbers but for a rounding of the sum (one half step of bf16 and fp32's)."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens = [40, 3, 0, 77]
    off = cu(np.concatenate([[0], np.cumsum(lens)]))
    x = rand((120, 4, 128), BF16, 8).cuda()
    tables = J.rotary_tables(128, 128)
    for inverse in (False, True):
        y, r = J.rotary(x, tables, off=off, inverse=inverse), J.rope(x, off, off, tables, inverse=inverse)
        within(y, np64(r), 2 * 2.0**-8 * np.abs(np64(r)) + 2.0**-20)
    assert J.device_status() == 0


def test_rotary_gradients():
    """The gradient is the transposed rotation: bit for bit rotary's own with inverse, and against differences, which are exact
    for a linear function but for rounding (x and its step are multiples of 2^-6 below 4: sums are exact; |y| below 12, u each)."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    cos, sin = angles(50, 20)
    t = (cu(cos), cu(sin))
    off, start = cu(np.array([0, 9, 33])), cu(np.array([2, 17]))
    for layout in ("interleaved", "half"):
        base = (rand((36, 3, 48), FP32, 1).clamp(-2, 2) * 64).round().div(64).cuda()
        x = base.clone().requires_grad_(True)
        dy = rand((36, 3, 48), FP32, 2).cuda()
        y = J.rotary(x, t, off=off, start=start, layout=layout)
        y.backward(dy)
        back = J.rotary(dy, t, off=off, start=start, layout=layout, inverse=True)
        assert torch.equal(x.grad, back) and bool((x.grad[33:] == 0).all())
        v = torch.zeros_like(base)
        v[4, 1, 7], v[30, 2, 45], v[20, 0, 0] = 1.0, -1.0, 0.5
        loss = lambda z: float((J.rotary(z, t, off=off, start=start, layout=layout).double() * dy.double()).sum())  # noqa: E731
        got = (loss(base + v) - loss(base - v)) / 2
        assert abs(got - float((back.double() * v.double()).sum())) <= 12 * 4 * R.U * 12 * float(dy.abs().max())
        x.grad = None
        J.rotary(x, t, off=off, start=start, layout=layout).sum().backward()  # an expanded gradient
        assert torch.equal(x.grad, J.rotary(torch.ones_like(dy), t, off=off, start=start, layout=layout, inverse=True))
    z = base.clone().requires_grad_(True)
    (gx,) = torch.autograd.grad(J.rotary(z, t, off=off).square().sum(), z, create_graph=True)
    gx.sum().backward()  # twice differentiable: it is linear
    assert bool(torch.isfinite(z.grad).all())
    assert J.device_status() == 0


def test_rotary_on_streams_and_in_graphs():
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    tables = J.rotary_tables(500, 64)
    x = rand((64, 6, 128), BF16, 1).cuda()
    start = torch.arange(64, device="cuda")
    out = torch.zeros_like(x)
    J.rotary(x, tables, start=start, layout="half", out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cos, sin = J.rotary_tables(500, 64, base=500.0)
        J.rotary(x, (cos, sin), start=start, layout="half", out=out)
    t2 = J.rotary_tables(500, 64, base=500.0)
    for t in range(5):
        start.add_(60)
        x.copy_(rand((64, 6, 128), BF16, 10 + t))
        graph.replay()
        assert torch.equal(out, J.rotary(x, t2, start=start, layout="half"))
    assert J.device_status() == 0


def test_rotary_python_refusals():
    import jagged_attention_recsys_gdpa_gb300 as J

    x = torch.zeros(6, 2, 64, dtype=BF16, device="cuda")
    c = torch.zeros(9, 32, device="cuda")
    i = torch.zeros(6, dtype=torch.int64, device="cuda")
    J.rotary(x, (c, c), start=i)
    for kw in (dict(x=x[0]), dict(x=x.double()), dict(x=x.cpu()), dict(x=x.transpose(1, 2)), dict(x=x[:, :0]), dict(x=x[..., :62]),
               dict(x=x[..., :1]), dict(cos=c.half()), dict(cos=c[:5]), dict(cos=c[0]), dict(cos=c.cpu()), dict(cos=c[:, ::2]),
               dict(start=i[:5]), dict(start=i.int()), dict(start=i.cpu()), dict(off=i, start=i), dict(off=i[:0], start=None),
               dict(off=i[:1], start=None), dict(off=i.int(), start=None), dict(layout="other"), dict(out=x.float()), dict(out=x[:3]),
               dict(out=x.clone().requires_grad_(True)), dict(x=x.clone().requires_grad_(True), out=x.clone()),
               dict(cos=c.clone().requires_grad_(True))):
        kw = dict(dict(x=x, cos=c, start=i), **kw)
        cos = kw.pop("cos")
        with pytest.raises(ValueError):
            J.rotary(kw.pop("x"), (cos, c), **kw)
    assert J.device_status() == 0


# ------------------------------------------------------------------ tables
@pytest.mark.parametrize("scaling,factor,original", [(None, 1.0, None), ("linear", 4.0, None), ("ntk", 8.0, None), ("yarn", 16.0, 4096),
                                                     ("yarn", 1.0, 100)])
@pytest.mark.parametrize("dim", [2, 4, 6, 64, 90, 128, 1024])
def test_rotary_tables(dim, scaling, factor, original):
    """Against 64 bits at near and far positions; cos and sin of the 64-bit angle are themselves exact to 2^-52 times it."""
    import jagged_attention_recsys_gdpa_gb300 as J

    if scaling == "ntk" and dim == 2:
        with pytest.raises(J.JattnError):
            J.rotary_tables(4, dim, scaling=scaling, factor=factor)
        return
    theta, size = R.theta(dim, 10000.0, scaling, factor, original)
    for first, rows in ((0, 1), (0, 300), (65_500, 77), (2**24 - 50, 50)):
        cos, sin = J.rotary_tables(rows, dim, scaling=scaling, factor=factor, original=original, first=first)
        ang = np.arange(first, first + rows)[:, None] * theta[None, :]
        within(cos, np.cos(ang) * size, 2.0**-22 * size)
        within(sin, np.sin(ang) * size, 2.0**-22 * size)


def test_rotary_tables_of_small_angles_keep_their_digits():
    """The slowest pairs' sines are tiny: relative to themselves they are within 2^-21 (the angle's float and the polynomial)."""
    import jagged_attention_recsys_gdpa_gb300 as J

    theta, _ = R.theta(256, 1e9)
    cos, sin = J.rotary_tables(2000, 256, base=1e9)
    ang = np.arange(2000)[:, None] * theta[None, :]
    slow = (ang < 0.7) & (ang > 0)
    assert np.all(np.abs(np64(sin) - np.sin(ang))[slow] <= 2.0**-21 * np.sin(ang)[slow])
    assert np.all(np64(sin)[0] == 0) and np.all(np64(cos)[0] == 1)


def test_rotary_tables_parts_and_shapes():
    import jagged_attention_recsys_gdpa_gb300 as J

    cos, sin = J.rotary_tables(100_003, 128)
    for first in (0, 7, 99_000):
        c, s = J.rotary_tables(1003, 128, first=first)
        assert torch.equal(c, cos[first:first + 1003]) and torch.equal(s, sin[first:first + 1003])
    c, s = J.rotary_tables(50_001, 126)
    assert c.shape == s.shape == (50_001, 63)
    empty, _ = J.rotary_tables(0, 64)
    assert empty.shape == (0, 32)
    # base and positions at the range's ends
    c, s = J.rotary_tables(3, 64, first=2**31 - 3)
    theta, _ = R.theta(64, 10000.0)
    ang = np.arange(2**31 - 3, 2**31)[:, None] * theta[None, :]
    # theta's own rounding and 2 pi's (2^-52 each, relative) times the position, for either side
    within(c, np.cos(ang), 2.0**-22 + 2 * 2.0**-51 * ang)


def test_rotary_tables_out_of_range_scalings():
    import jagged_attention_recsys_gdpa_gb300 as J

    for kw in (dict(base=1.0), dict(base=float("inf")), dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=2.0, original=-5),
               dict(scaling="yarn", factor=2.0, original=100, beta_fast=1.0), dict(scaling="ntk", factor=1e300)):
        with pytest.raises(J.JattnError):
            J.rotary_tables(4, 64, **kw)
    assert ctypes.sizeof(J._binding.RotaryTables) == 8 * 2 + 4 * 2 + 8 * 5
