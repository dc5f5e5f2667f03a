"""Plain 64-bit references of layer norm, rotary positions and their tables, and
of the page pool, written from their definitions, with the bounds that the
arithmetic gives."""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0**-24  # half a step of fp32, relative
HALF_STEP = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float32: 2.0**-24}
# half a step below the normal numbers, where the relative half step is too small
TINY = {torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25, torch.float32: 2.0**-150}


def np64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ layer norm
def layer_norm(x, w, b, eps):
    """(y, mean, rstd) of float64 rows [..., N]."""
    m = x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - m) * rstd
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, m[..., 0], rstd[..., 0]


def layer_norm_bounds(x, w, b, eps, dtype):
    """Bounds of (y, mean, rstd) for sums held in fp32, u = 2^-24.

    A sum of N terms goes through at most 16 additions in a lane and 10 across lanes: 26 u of the terms' sizes, with the
    division 28 u. With m~ the rounded mean, |m~ - m| <= 28 u mean|x| = e; the differences x - m~ are rounded once each. Their mean
    corrects m~: what is left of the error is 30 u of mean|x - m~| <= mean|x - m| + e. The variance is off by 30 u of mean (x - m~)^2 = v + e^2
    (its terms, their sum, the correction), so rstd by half of that over v + eps, 2^-22 for the reciprocal root
    and u for eps. y takes both, the products' and the sum's roundings (4 u) and the rounding to its type."""
    m = x.mean(-1, keepdims=True)
    e = 28 * U * np.abs(x).mean(-1, keepdims=True)
    v = ((x - m) ** 2).mean(-1, keepdims=True)
    spread = np.abs(x - m).mean(-1, keepdims=True) + e
    d_err = 30 * U * spread + 2 * U * (np.abs(x - m) + e)
    rstd = 1.0 / np.sqrt(v + eps)
    r_rel = 15 * U * (v + e**2) / (v + eps) + 4 * U + 2 * U
    h = np.abs(x - m) * rstd
    scale = 1.0 if w is None else np.abs(w)
    shift = 0.0 if b is None else np.abs(b)
    y = layer_norm(x, w, b, eps)[0]
    y_err = scale * (d_err * rstd + h * r_rel) + 4 * U * (scale * h + shift)
    y_err = y_err + HALF_STEP[dtype] * (np.abs(y) + y_err) + TINY[dtype]
    mean_err = 30 * U * spread + 2 * U * np.abs(m)
    return y_err, mean_err[..., 0], (rstd * r_rel)[..., 0]


def layer_norm_grads(dy, x, w, rstd):
    """(dx, dw, db) of float64 rows, h from x's own mean and the given rstd [...]."""
    h = (x - x.mean(-1, keepdims=True)) * rstd[..., None]
    g = dy if w is None else dy * w
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - h * (g * h).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, (dy * h).sum(axes), dy.sum(axes)


def layer_norm_grad_bounds(dy, x, w, rstd, dtype, weight_dtype, depth):
    """Bounds of (dx, dw, db), u = 2^-24; the sums over a row as above (28 u with their division). The given mean is off by o = 2 u|m| (and 30 u of
    the spread), its correction by 30 u of mean|x - m| + o (each difference is rounded): h is off by eh = rstd (30 u (mean|x - m| + o) +
    2 u (|x - m| + o)) + 2 u |h|. g = dy w: u. mean(g): 29 u mean|g|. mean(g h) = rstd (sum g d - c sum g) / N: 30 u of
    mean(|g| (|h| + rstd (mean|x - m| + o))). dx: those, and 4 u of each term.
    A sum over rows takes `depth` additions and each term's own error."""
    m = x.mean(-1, keepdims=True)
    r = rstd[..., None]
    g = np.abs(dy) if w is None else np.abs(dy * w)
    off = 2 * U * np.abs(m) + 30 * U * np.abs(x - m).mean(-1, keepdims=True)
    spread = np.abs(x - m).mean(-1, keepdims=True) + off
    h = np.abs(x - m) * r
    eh = r * (30 * U * spread + 2 * U * (np.abs(x - m) + off)) + 2 * U * h
    mg = g.mean(-1, keepdims=True)
    mgh_size = (g * (h + r * (spread + off))).mean(-1, keepdims=True)
    dx, dw, db = layer_norm_grads(dy, x, w, rstd)
    e = r * (4 * U * g + 33 * U * mg + 36 * U * h * mgh_size + eh * mgh_size)
    e = e + HALF_STEP[dtype] * (np.abs(dx) + e) + TINY[dtype]
    axes = tuple(range(x.ndim - 1))
    ew = (np.abs(dy) * (eh + U * h)).sum(axes) + depth * U * (np.abs(dy) * (h + eh)).sum(axes)
    eb = depth * U * np.abs(dy).sum(axes)
    half, tiny = HALF_STEP[weight_dtype], TINY[weight_dtype]
    return e, ew + half * (np.abs(dw) + ew) + tiny, eb + half * (np.abs(db) + eb) + tiny


# ------------------------------------------------------------------ rotary positions
def positions(total, off, start):
    """Each row's position, -1 for rows that are skipped."""
    if off is None:
        return np.arange(total) if start is None else np.where(start < 0, -1, start)
    pos = np.full(total, -1)
    for b in range(len(off) - 1):
        s = 0 if start is None else start[b]
        if s >= 0:
            pos[off[b]:off[b + 1]] = s + np.arange(off[b + 1] - off[b])
    return pos


def rotary(x, cos, sin, pos, layout, inverse):
    """x (a CPU tensor [total, H, D]) rotated in fp32, every product and sum rounded by itself, and rounded once to its
    type; rows of negative positions zero, rows behind the tables as they are."""
    half = cos.shape[1]
    f = x.float().numpy()
    turn = (pos >= 0) & (pos < cos.shape[0])
    at = np.where(turn, pos, 0)
    c, s = cos[at][:, None, :], sin[at][:, None, :] * np.float32(-1 if inverse else 1)
    if layout == "half":
        ia, ib = np.arange(half), np.arange(half) + half
    else:
        ia, ib = 2 * np.arange(half), 2 * np.arange(half) + 1
    y = f.copy()
    a, b = f[..., ia], f[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    y = np.where(turn[:, None, None], y, f)
    y = np.where((pos < 0)[:, None, None], np.float32(0), y)
    return torch.from_numpy(y).to(x.dtype)


def theta(dim, base, scaling=None, factor=1.0, original=None, beta_fast=32.0, beta_slow=1.0):
    """(angle per position of each pair, amplitude) in 64 bits."""
    out = []
    for m in range(dim // 2):
        b = base * factor ** (dim / (dim - 2)) if scaling == "ntk" else base
        t = b ** (-2 * m / dim)
        if scaling == "linear":
            t = t / factor
        if scaling == "yarn":
            turns = original * t / (2 * math.pi)
            keep = min(max((turns - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0)
            t = (1 - keep) * t / factor + keep * t
        out.append(t)
    return np.array(out), 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0


# ------------------------------------------------------------------ page pool
class Pool:
    """The pool as a list, one page after another."""

    def __init__(self, n_pages, page):
        self.free, self.n, self.page = list(range(n_pages - 1, -1, -1)), n_pages, page

    def _pages(self, rows):
        return -(-rows // self.page)

    def assign(self, table, start, lens, total):
        """table is changed; the slots of all rows, in order. None where the pool is short."""
        B, P = table.shape
        wanted = []
        ok = [start[b] >= 0 and start[b] + lens[b] <= P * self.page for b in range(B)]
        for b in range(B):
            if ok[b]:
                wanted += [(b, j) for j in range(self._pages(start[b]), self._pages(start[b] + lens[b]))]
        if len(wanted) > len(self.free):
            return None
        for b, j in wanted:
            table[b, j] = self.free.pop()
        slots, r = np.full(total, -1, np.int64), 0
        for b in range(B):
            for i in range(lens[b]):
                if ok[b]:
                    pos = start[b] + i
                    slots[r] = int(table[b, pos // self.page]) * self.page + pos % self.page
                r += 1
        return slots

    def release(self, table, lens, keep):
        back = []
        for b in range(len(lens)):
            k = 0 if keep is None else keep[b]
            if k < 0 or lens[b] <= k or lens[b] > table.shape[1] * self.page:
                continue
            js = range(self._pages(k), self._pages(lens[b]))
            if any(not 0 <= table[b, j] < self.n for j in js):
                continue
            back += [(b, j) for j in js]
        if len(back) + len(self.free) > self.n:
            return False
        self.free += [int(table[b, j]) for b, j in reversed(back)]
        for b, j in back:
            table[b, j] = -1
        return True
