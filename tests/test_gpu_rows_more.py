"""Row operators where the tests of each operator's range do not reach: derivatives in forward mode and traces, statistics
of padding and of rows that are not finite, and every number of heads that a thread of the rotation takes."""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from tests import rows_ref as R
from tests.rows_ref import np64
from tests.test_gpu_rows import BF16, FP16, FP32, TYPES, clear, cu, rand, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ statistics
def poisoned(n):
    """Memory that the next calls' outputs are likely to get: NaN."""
    blocks = [torch.full((n,), float("nan"), device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("n", [128, 100, 1001])
@pytest.mark.parametrize("heads", [1, 3])
def test_statistics_of_padding_are_zero(n, heads):
    """mean and rstd are outputs that the call allocates: zero behind the last sequence, also where y is the caller's and its
    padding stays as it was."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    for live, total in ((0, 5), (29, 40), (100, 300), (40, 40)):
        off = cu(np.array([0, live // 2, live]))
        x = rand((total, heads, n), BF16, 1).cuda()
        out = torch.full_like(x, 5.0)
        want = J.layer_norm_forward(x, off=off)
        for _ in range(4):
            poisoned(2 * (-(-total * heads // 64) * 64))
            y, mean, rstd = J.layer_norm_forward(x, off=off, out=out)
            assert torch.equal(mean, want[1]) and torch.equal(rstd, want[2])
            assert bool((mean[live:] == 0).all()) and bool((rstd[live:] == 0).all())
            assert bool((y[live:] == 5.0).all()) and torch.equal(y[:live], want[0][:live])
    assert J.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 7, 64, 100, 1001, 2048, 9000])
def test_statistics_of_rows_that_are_not_finite(n, dtype):
    """The formulas' own: a NaN makes both NaN, an infinity is its row's mean and leaves no spread that is a number."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    inf, nan = float("inf"), float("nan")
    x = rand((6, n), dtype, 1)
    x[1, n // 2], x[2, n - 1], x[3, 0], x[4, :] = nan, inf, -inf, inf
    y, mean, rstd = J.layer_norm_forward(x.cuda())
    want = x.double().mean(-1).numpy()
    got = np64(mean)
    assert np.isnan(got[1]) and got[2] == inf and got[3] == -inf and got[4] == inf
    assert np.isfinite(got[[0, 5]]).all() and np.isfinite(want[[0, 5]]).all()
    assert bool(torch.isnan(rstd[1:5]).all()) and bool(torch.isfinite(rstd[[0, 5]]).all())
    assert bool(torch.isnan(y[1:5]).all()) and bool(torch.isfinite(y[[0, 5]]).all())
    dx, _, _ = J.layer_norm_backward(x.cuda(), x.cuda(), None, mean, rstd)
    assert bool(torch.isnan(dx[1:5]).all()) and bool(torch.isfinite(dx[[0, 5]]).all())
    assert J.device_status() == 0


# ------------------------------------------------------------------ derivatives of the rotation
def rotations():
    """Tables and positions of 40 rows: padding, a sequence that is skipped, positions behind the tables."""
    a = np.random.default_rng(1).uniform(-4, 4, (50, 20))
    t = (cu(np.cos(a).astype(np.float32)), cu(np.sin(a).astype(np.float32)))
    return t, cu(np.array([0, 9, 20, 33])), cu(np.array([2, -1, 45]))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_carries_tangents(layout, inverse):
    """Forward mode: the rotation is linear, so the tangent is the rotated tangent, bit for bit, whatever the grad mode."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    t, off, start = rotations()
    x, dx = rand((40, 3, 48), FP32, 1).cuda(), rand((40, 3, 48), FP32, 2).cuda()

    def turn(z):
        return J.rotary(z, t, off=off, start=start, layout=layout, inverse=inverse)

    y, dy = turn(x), turn(dx)
    for grad in (True, False):
        for leaf in (False, True):
            with torch.set_grad_enabled(grad), fwAD.dual_level():
                z = x.clone().requires_grad_(leaf)
                p, v = fwAD.unpack_dual(turn(fwAD.make_dual(z, dx)))
                assert torch.equal(p, y) and v is not None and torch.equal(v, dy)
    with torch.no_grad(), fwAD.dual_level():  # an expanded tangent, and part of a fused tensor
        p, v = fwAD.unpack_dual(turn(fwAD.make_dual(x, torch.ones((), device="cuda").expand_as(x))))
        assert torch.equal(p, y) and torch.equal(v, turn(torch.ones_like(x)))
        fused = fwAD.make_dual(torch.cat([x, x], 1), torch.cat([dx, dx], 1))
        p, v = fwAD.unpack_dual(turn(fused[:, 3:]))
        assert torch.equal(p, y) and torch.equal(v, dy)
    with fwAD.dual_level():  # the gradient of a gradient's direction: R' (2 R dx)
        z = x.clone().requires_grad_(True)
        (g,) = torch.autograd.grad(turn(fwAD.make_dual(z, dx)).square().sum(), z)
        back = J.rotary(2 * dy, t, off=off, start=start, layout=layout, inverse=not inverse)
        assert torch.equal(fwAD.unpack_dual(g).tangent, back)
    with fwAD.dual_level():
        z = fwAD.make_dual(x.clone(), dx)
        for out in (torch.empty_like(x), z):
            with pytest.raises(ValueError):
                J.rotary(z, t, off=off, start=start, out=out)
        turning = (fwAD.make_dual(t[0], torch.ones_like(t[0])), t[1])
        for rows in (x, z, x.clone().requires_grad_(True)):
            with pytest.raises(ValueError):
                J.rotary(rows, turning, off=off, start=start)
            with pytest.raises(ValueError):
                J.rotary(rows, turning[::-1], off=off, start=start)
        with pytest.raises(RuntimeError):  # layer norm has no forward mode, and says so
            J.layer_norm(z)
        assert torch.equal(turn(x), y)  # rows without a tangent are as ever
    J.device_status()


def test_rotary_twice_differentiated():
    """The gradient of sum(g(z)), g the gradient of sum(y^2): R' 2 R 1, bit for bit what the calls give one after another."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    t, off, start = rotations()
    for layout in ("interleaved", "half"):
        z = rand((40, 3, 48), FP32, 1).cuda().requires_grad_(True)
        y = J.rotary(z, t, off=off, start=start, layout=layout)
        (g,) = torch.autograd.grad(y.square().sum(), z, create_graph=True)
        assert torch.equal(g, J.rotary(2 * y.detach(), t, off=off, start=start, layout=layout, inverse=True))
        g.sum().backward()
        ones = J.rotary(torch.ones_like(y), t, off=off, start=start, layout=layout)
        assert torch.equal(z.grad, J.rotary(2 * ones, t, off=off, start=start, layout=layout, inverse=True))
    J.device_status()


@pytest.mark.filterwarnings("ignore")
def test_rotary_is_recorded_by_a_trace():
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    t, off, _ = rotations()
    x, other = rand((40, 3, 48), FP32, 1).cuda(), rand((40, 3, 48), FP32, 2).cuda()
    traced = torch.jit.trace(lambda z: J.rotary(z, t, off=off), x, check_trace=False)
    assert torch.equal(traced(other), J.rotary(other, t, off=off))
    J.device_status()
