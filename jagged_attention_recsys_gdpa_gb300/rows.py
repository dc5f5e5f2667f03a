"""Rows on their way to attention: layer norm and rotary positions.

* ``layer_norm(x, weight, bias, eps=..., off=...)``: layer norm over the last
  dimension with autograd; ``layer_norm_forward`` -> (y, mean, rstd) and
  ``layer_norm_backward`` -> (dx, dweight, dbias): the raw passes. Query/key norm is
  a layer norm of [total, H, D] rows with a weight of D values.
* ``rotary(x, tables, off=..., start=..., layout=..., inverse=...)``: rotary
  positions in either layout, on all of a head's columns or the first ones, with
  autograd. ``rope`` rotates the same pairs of neighbours for ``attention`` and
  ``backward``, at positions that two offset lists give.
* ``rotary_tables(rows, dim, base=..., scaling=...)``: the cos and sin tables for
  ``rotary``, ``rope``, ``attention`` and ``cache_append``, scaled for long contexts.

Rows are bf16, fp16 or fp32 CUDA tensors [total, H, D] (layer norm: or [rows, N])
whose last dimension is dense; the others may have any strides, so heads of a fused
projection need no copy. Sums and products are held in fp32 and results rounded
once. Calls run on the current stream of the tensors' device and allocate only
outputs and scratch, from PyTorch's allocator. With ``off`` (int64 prefix sums), rows behind
off[-1] are padding: zero in outputs that a call allocates, left as they were in those it
is given, and in no sum. Device-side errors are read with ``device_status``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as B
from .paged import _C_device, _C_stream, _check_no_grad, _status_address, _status_addresses

_TYPES = {torch.float32: B.F32, torch.bfloat16: B.BF16, torch.float16: B.F16}
_LAYOUTS = {"interleaved": B.ROTARY_INTERLEAVED, "half": B.ROTARY_HALF}
_SCALINGS = {None: B.SCALE_NONE, "none": B.SCALE_NONE, "linear": B.SCALE_LINEAR, "ntk": B.SCALE_NTK,
             "yarn": B.SCALE_YARN}

# What a call derives from sizes, strides, types and the device alone, kept for the next call of the same ones: checked
# arguments as a C structure, and sizes of what it allocates. Dropped as a whole when a program shows ever new sizes.
_plans: dict = {}
_MOST_PLANS = 4096


def _keep(key, plan):
    if len(_plans) >= _MOST_PLANS:
        _plans.clear()
    _plans[key] = plan
    return plan


def _elsewhere(index, call, *args, **kw):
    """call(*args, **kw) with the device of its tensors current."""
    with torch.cuda.device(index):
        return call(*args, **kw)


def _strides(x, name):
    """(row stride, head stride) of x [rows, N] or [rows, heads, N]; those of dimensions of one entry as in a dense one."""
    dims = x.dim()
    if x.dtype not in _TYPES or not x.is_cuda or dims < 2 or dims > 3:
        raise ValueError(f"{name} must be a CUDA tensor [rows, N] or [rows, heads, N] of bf16, fp16 or fp32")
    shape, strides = x.shape, x.stride()
    n = shape[-1]
    if strides[-1] != 1 and n > 1:
        raise ValueError(f"the values of a row of {name} must be neighbours in memory")
    head = strides[1] if dims == 3 and shape[1] > 1 else n
    heads = shape[1] if dims == 3 else 1
    return (strides[0] if shape[0] > 1 else heads * head), head


def _like(t, x, name):
    if t.dtype is not x.dtype or t.shape != x.shape or t.device != x.device:
        raise ValueError(f"{name} must have x's shape, type and device")


def _live(x, off):
    """Address of the number of rows that are no padding."""
    if off is None:
        return None
    if off.dtype is not torch.int64 or off.dim() != 1 or off.numel() < 1 or off.device != x.device \
            or not off.is_contiguous():
        raise ValueError("off must be a contiguous int64 tensor [B+1] on x's device")
    return off.data_ptr() + 8 * (off.numel() - 1)


def _check_weight(x, w, name):
    if w.shape != x.shape[-1:] or w.device != x.device or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor [N] of x's type or fp32 on x's device")


def _check_stats(x, t, shape, name):
    if t.dtype is not torch.float32 or t.shape != shape or t.device != x.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor of x's shape without its last dimension")


def _norm_plan(x, weight, eps, dy, out):
    """(C structure, the statistics' shape, bytes of scratch) for x's sizes; dy: of the backward, else None."""
    key = (x.shape, x.stride(), x.dtype, x.device, None if weight is None else weight.dtype, eps,
           None if dy is None else dy.stride(), None if out is None else out.stride())
    plan = _plans.get(key)
    if plan is not None:
        return plan
    xs = _strides(x, "x")
    n, heads = x.shape[-1], x.shape[1] if x.dim() == 3 else 1
    if not 1 <= n <= 16384 or heads < 1:
        raise ValueError("rows must have 1 to 16384 values, and at least one head")
    if weight is not None and weight.dtype not in (x.dtype, torch.float32):
        raise ValueError("weight must have x's type or fp32")
    if not 0.0 < eps < float("inf"):
        raise ValueError("eps must be positive and finite")
    t = _TYPES[x.dtype]
    two = ctypes.c_int64 * 2
    ys = (heads * n, n) if out is None else _strides(out, "out")
    p = ctypes.byref(B.Norm(x.shape[0], heads, n, t, t if weight is None else _TYPES[weight.dtype], eps, int(out is None),
                            two(*xs), two(*ys), two(*((0, 0) if dy is None else _strides(dy, "dy")))))
    scratch = 0
    if dy is not None and weight is not None:
        with torch.cuda.device(x.device):
            scratch = B.layer_norm_bwd_scratch_size(p)
    return _keep(key, (p, x.shape[:-1], scratch))


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, off=None, out=None):
    """y = (x - mean) rstd weight + bias over the last dimension, rstd = 1 / sqrt(variance + eps). Returns (y, mean, rstd), the
    statistics fp32 of x's shape without its last dimension. weight and bias are [N] of x's type or fp32 (None: ones and
    zeros). ``out`` may be x. See jattn_layer_norm."""
    if out is not None:
        _like(out, x, "out")
        _check_no_grad(out)
    p, stats, _ = _norm_plan(x, weight, eps, None, out)
    w = b = None
    if weight is not None:
        _check_weight(x, weight, "weight")
        w = weight.data_ptr()
    if bias is not None:
        if weight is None or bias.dtype is not weight.dtype:
            raise ValueError("a bias needs a weight of its type")
        _check_weight(x, bias, "bias")
        b = bias.data_ptr()
    live = None if off is None else _live(x, off)
    dev = x.device
    index = dev.index
    if _C_device() != index:
        return _elsewhere(index, layer_norm_forward, x, weight, bias, eps, off, out)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    mean = torch.empty(stats, dtype=torch.float32, device=dev)
    rstd = torch.empty(stats, dtype=torch.float32, device=dev)
    rc = (B._lib or B.load()).jattn_layer_norm(
        p, live, x.data_ptr(), w, b, out.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        _status_addresses.get(index) or _status_address(index), 256, _C_stream(index))
    if rc:
        B.check(rc, "jattn_layer_norm")
    return out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, off=None, bias=True, out=None):
    """Gradients (dx, dweight, dbias) of layer_norm_forward from its statistics; dweight and dbias (None without weight, or with
    ``bias`` False) are summed over all rows in fp32 and have weight's type. ``out`` (dx) may be dy or x. See
    jattn_layer_norm_bwd."""
    _like(dy, x, "dy")
    if out is not None:
        _like(out, x, "out")
        _check_no_grad(out)
    p, stats, n = _norm_plan(x, weight, 1.0, dy, out)
    _check_stats(x, mean, stats, "mean")
    _check_stats(x, rstd, stats, "rstd")
    live = None if off is None else _live(x, off)
    dev = x.device
    index = dev.index
    if _C_device() != index:
        return _elsewhere(index, layer_norm_backward, dy, x, weight, mean, rstd, off, bias, out)
    w = dw = db = scratch = None
    if weight is not None:
        _check_weight(x, weight, "weight")
        w = weight.data_ptr()
        dw = torch.empty_like(weight)
        db = torch.empty_like(weight) if bias else None
        scratch = torch.empty(n, dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    rc = (B._lib or B.load()).jattn_layer_norm_bwd(
        p, live, dy.data_ptr(), x.data_ptr(), w, mean.data_ptr(), rstd.data_ptr(), out.data_ptr(), B.ptr(dw), B.ptr(db),
        B.ptr(scratch), n, _status_addresses.get(index) or _status_address(index), 256, _C_stream(index))
    if rc:
        B.check(rc, "jattn_layer_norm_bwd")
    return out, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, off):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps, off)
        ctx.save_for_backward(x, weight, mean, rstd, off)
        ctx.bias = bias is not None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd, off = ctx.saved_tensors
        if dy.stride(-1) != 1:
            dy = dy.contiguous()
        learns = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        if weight is not None and not learns and not ctx.needs_input_grad[0]:
            return None, None, None, None, None
        dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd, off, ctx.needs_input_grad[2])
        return dx, dw if ctx.needs_input_grad[1] else None, db, None, None


def layer_norm(x, weight=None, bias=None, eps=1e-5, off=None):
    """Layer norm over the last dimension with autograd: gradients for x, weight and bias. See layer_norm_forward."""
    return _LayerNorm.apply(x, weight, bias, eps, off)


def _rotary_plan(x, cos, nb, layout, inverse, out):
    key = (x.shape, x.stride(), x.dtype, x.device, cos.shape, nb, layout, inverse, None if out is None else out.stride())
    plan = _plans.get(key)
    if plan is not None:
        return plan
    if x.dim() != 3:
        raise ValueError("x must be [total, H, D]")
    xs = _strides(x, "x")
    total, heads, D = x.shape
    if cos.dim() != 2 or not 1 <= cos.shape[1] <= D // 2 or not 2 <= D <= 16384 or heads < 1:
        raise ValueError("tables must have 1 to D/2 columns, and x at least one head of 2 to 16384 columns")
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}")
    two = ctypes.c_int64 * 2
    ys = (heads * D, D) if out is None else _strides(out, "out")
    return _keep(key, ctypes.byref(B.Rotary(nb, total, heads, D, cos.shape[1], _TYPES[x.dtype], _LAYOUTS[layout], inverse,
                                            int(out is None), cos.shape[0], two(*xs), two(*ys))))


def _rotate(x, cos, sin, off, start, layout, inverse, out):
    dev = x.device
    for t in (off, start):
        if t is not None and (t.dtype is not torch.int64 or t.dim() != 1 or t.device != dev or not t.is_contiguous()):
            raise ValueError("off and start must be contiguous int64 tensors on x's device")
    nb = x.shape[0] if off is None else off.numel() - 1
    if nb < (off is not None) or (start is not None and start.numel() != nb):
        raise ValueError("start must have an entry per sequence of off, or per row without off")
    p = _rotary_plan(x, cos, nb, layout, inverse, out)
    index = dev.index
    if _C_device() != index:
        return _elsewhere(index, _rotate, x, cos, sin, off, start, layout, inverse, out)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    rc = (B._lib or B.load()).jattn_rotary(
        p, None if off is None else off.data_ptr(), None if start is None else start.data_ptr(), cos.data_ptr(),
        sin.data_ptr(), x.data_ptr(), out.data_ptr(), _status_addresses.get(index) or _status_address(index), 256,
        _C_stream(index))
    if rc:
        B.check(rc, "jattn_rotary")
    return out


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, cos, sin, off, start, layout, inverse):
        ctx.save_for_backward(cos, sin, off, start)
        ctx.how = layout, inverse
        return _rotate(x, cos, sin, off, start, layout, inverse, None)

    @staticmethod
    def backward(ctx, dy):
        cos, sin, off, start = ctx.saved_tensors
        layout, inverse = ctx.how
        if dy.stride(-1) != 1:
            dy = dy.contiguous()
        return _Rotary.apply(dy, cos, sin, off, start, layout, not inverse), None, None, None, None, None, None


def rotary(x, tables, off=None, start=None, layout="interleaved", inverse=False, out=None):
    """Rotary positions of rows x [total, H, D]: with ``tables`` = (cos, sin) fp32 [rows, R/2], R <= D, the pairs of the
    first R columns of every head, (2m, 2m + 1) in layout "interleaved" or (m, m + R/2) in layout "half", turn by the angles
    of the row's position (back, with ``inverse``); the other columns stay. Row i of sequence b (``off`` int64 [B+1])
    stands at start[b] + i (``start`` int64 [B], None: 0); without off row r stands at start[r] (int64 [total], None: r).
    A negative start skips its rows as padding is. ``out`` may be x. With autograd (the gradient turns back), but for ``out``.
    See jattn_rotary."""
    cos, sin = tables
    for t in tables:
        if t.dtype is not torch.float32 or t.shape != cos.shape or t.device != x.device or not t.is_contiguous():
            raise ValueError("tables must be two contiguous fp32 tensors [rows, R/2] on x's device")
    if torch.is_grad_enabled():
        if cos.requires_grad or sin.requires_grad:
            raise ValueError("tables take no gradient: pass detached tensors")
        if x.requires_grad:
            if out is not None:
                raise ValueError("out is written without a gradient: call under torch.no_grad() or on a detached x")
            return _Rotary.apply(x, cos, sin, off, start, layout, bool(inverse))
    if out is not None:
        _like(out, x, "out")
        _check_no_grad(out)
    return _rotate(x, cos, sin, off, start, layout, bool(inverse), out)


def rotary_tables(rows, dim, base=10000.0, scaling=None, factor=1.0, original=None, beta_fast=32.0, beta_slow=1.0, first=0,
                  device="cuda"):
    """(cos, sin) fp32 [rows, dim/2] of positions first .. first + rows - 1: angle pos * theta_m, theta_m = base^(-2m/dim).
    ``scaling`` for contexts ``factor`` times as long as the model was trained on: "linear" (theta_m / factor), "ntk" (a larger base) or "yarn"
    (fast pairs as they are, slow ones / factor, by their turns within ``original`` positions, and values times 0.1
    ln(factor) + 1). Angles are exact to 2^-53 of theta however far the position lies. See jattn_rotary_tables."""
    dev = torch.device(device)
    key = (rows, dim, base, scaling, factor, original, beta_fast, beta_slow, first)
    plan = _plans.get(key)
    if plan is None:
        if scaling not in _SCALINGS:
            raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
        if dim < 2 or dim % 2 or dim > 1024:
            raise ValueError("dim must be even, from 2 to 1024")
        if rows < 0 or first < 0 or first + rows > 1 << 31:
            raise ValueError("positions must lie between 0 and 2^31")
        if scaling == "yarn" and original is None:
            raise ValueError("yarn needs the original context")
        plan = _keep(key, ctypes.byref(B.RotaryTables(first, rows, dim // 2, _SCALINGS[scaling], base, factor,
                                                      original or 0.0, beta_fast, beta_slow)))
    if dev.type != "cuda":
        raise ValueError("tables are made on a CUDA device")
    cos = torch.empty((rows, dim // 2), dtype=torch.float32, device=dev)
    sin = torch.empty((rows, dim // 2), dtype=torch.float32, device=dev)
    index = cos.device.index
    if _C_device() != index:
        return _elsewhere(index, rotary_tables, rows, dim, base, scaling, factor, original, beta_fast, beta_slow, first, cos.device)
    rc = (B._lib or B.load()).jattn_rotary_tables(plan, cos.data_ptr(), sin.data_ptr(), _C_stream(index))
    if rc:
        B.check(rc, "jattn_rotary_tables")
    return cos, sin
