"""Rows on their way to attention: layer norm and rotary positions.

* ``layer_norm(x, weight, bias, eps=..., off=...)``: layer norm over the last
  dimension with autograd; ``layer_norm_forward`` -> (y, mean, rstd) and
  ``layer_norm_backward`` -> (dx, dweight, dbias): the raw passes, which autograd does
  not follow. Query/key norm is a layer norm of [total, H, D] rows with a weight of D
  values. There is no forward mode (a tangent is refused) and no second derivative.
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

import torch

from . import _binding as B

_LAYOUTS = {"interleaved": B.ROTARY_INTERLEAVED, "half": B.ROTARY_HALF}
_SCALINGS = {None: B.SCALE_NONE, "none": B.SCALE_NONE, "linear": B.SCALE_LINEAR, "ntk": B.SCALE_NTK,
             "yarn": B.SCALE_YARN}


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, off=None, out=None):
    """y = (x - mean) rstd weight + bias over the last dimension, rstd = 1 / sqrt(variance + eps). Returns (y, mean, rstd), the
    statistics fp32 of x's shape without its last dimension. weight and bias are [N] of x's type or fp32 (None: ones and
    zeros). ``out`` may be x. See jattn_layer_norm."""
    return (B._host or B.host()).layer_norm(x, weight, bias, eps, off, out)


def layer_norm_backward(dy, x, weight, mean, rstd, off=None, bias=True, out=None):
    """Gradients (dx, dweight, dbias) of layer_norm_forward from its statistics; dweight and dbias (None without weight, or with
    ``bias`` False) are summed over all rows in fp32 and have weight's type. ``out`` (dx) may be dy or x. See
    jattn_layer_norm_bwd."""
    return (B._host or B.host()).layer_norm_bwd(dy, x, weight, mean, rstd, off, bias, out)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, off):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps, off)
        ctx.save_for_backward(x, weight, mean, rstd, off)
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


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, cos, sin, off, start, layout, inverse):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(cos, sin, off, start)
        ctx.save_for_forward(cos, sin, off, start)
        ctx.how = layout, inverse
        return B.host().rotary(x, cos, sin, off, start, layout, inverse, None)

    @staticmethod
    def backward(ctx, dy):
        return _Rotary._turn(ctx, dy, True), None, None, None, None, None, None

    @staticmethod
    def jvp(ctx, dx, dcos, dsin, *others):
        if dcos is not None or dsin is not None:
            raise ValueError("tables take no gradient: pass detached tensors")
        return _Rotary._turn(ctx, dx, False)

    @staticmethod
    def _turn(ctx, d, back):
        """A gradient turned back, or a tangent turned as the rows are."""
        if d is None:
            return None
        cos, sin, off, start = ctx.saved_tensors
        layout, inverse = ctx.how
        if d.stride(-1) != 1:
            d = d.contiguous()
        return _Rotary.apply(d, cos, sin, off, start, layout, inverse != back)


def rotary(x, tables, off=None, start=None, layout="interleaved", inverse=False, out=None):
    """Rotary positions of rows x [total, H, D]: with ``tables`` = (cos, sin) fp32 [rows, R/2], R <= D, the pairs of the
    first R columns of every head, (2m, 2m + 1) in layout "interleaved" or (m, m + R/2) in layout "half", turn by the angles
    of the row's position (back, with ``inverse``); the other columns stay. Row i of sequence b (``off`` int64 [B+1])
    stands at start[b] + i (``start`` int64 [B], None: 0); without off row r stands at start[r] (int64 [total], None: r).
    A negative start skips its rows as padding is. ``out`` may be x. With autograd in both modes (the gradient turns back, a
    tangent as the rows do) and in traces, but for ``out``. See jattn_rotary."""
    cos, sin = tables
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}")
    host = B._host or B.host()
    if host.rotary_followed(x, cos, sin):
        if out is not None:
            raise ValueError("out is written without a gradient: call under torch.no_grad() or on a detached x")
        return _Rotary.apply(x, cos, sin, off, start, _LAYOUTS[layout], bool(inverse))
    return host.rotary(x, cos, sin, off, start, _LAYOUTS[layout], inverse, out)


def rotary_tables(rows, dim, base=10000.0, scaling=None, factor=1.0, original=None, beta_fast=32.0, beta_slow=1.0, first=0,
                  device="cuda"):
    """(cos, sin) fp32 [rows, dim/2] of positions first .. first + rows - 1: angle pos * theta_m, theta_m = base^(-2m/dim).
    ``scaling`` for contexts ``factor`` times as long as the model was trained on: "linear" (theta_m / factor), "ntk" (a larger base) or "yarn"
    (fast pairs as they are, slow ones / factor, by their turns within ``original`` positions, and values times 0.1
    ln(factor) + 1; the ramp between ``beta_slow`` and ``beta_fast`` is linear in the turns, the paper's, not in the pair's index
    as in some programs). Angles are exact to 2^-53 of theta however far the position lies. See jattn_rotary_tables."""
    if scaling not in _SCALINGS:
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    if scaling == "yarn" and original is None:
        raise ValueError("yarn needs the original context")
    index = -1  # the current device
    if device != "cuda":
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("tables are made on a CUDA device")
        index = -1 if device.index is None else device.index
    return (B._host or B.host()).rotary_tables(rows, dim, base, _SCALINGS[scaling], factor, original or 0.0, beta_fast,
                                               beta_slow, first, index)
