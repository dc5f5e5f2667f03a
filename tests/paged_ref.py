"""Plain 64-bit reference of the paged-cache operators (numpy / torch on the
CPU), written from their definitions: page lookups one position at a time,
quantisation by searching the E4M3 grid, attention row by row."""
from __future__ import annotations

import math

import numpy as np
import torch

ACTS = ("softmax", "silu", "gelu", "gelu_poly")

# the finite E4M3 values of codes 0 .. 126 (sign bit clear)
E4M3 = np.array([(c & 7) * 2.0**-9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def e4m3_codes(x):
    """Nearest E4M3 codes of a float64 array (ties to the even code, saturated)."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    up = (a - E4M3[lo] > E4M3[hi] - a) | ((a - E4M3[lo] == E4M3[hi] - a) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return code | np.where(np.signbit(x), 128, 0).astype(np.uint8)


def e4m3_values(codes):
    return np.where(codes & 128, -1.0, 1.0) * np.append(E4M3, np.nan)[codes & 127]


def quantise(x):
    """float64 rows [..., D] -> (codes, exponents): one exponent per 32 neighbours, 255 for a block with NaN / Inf."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    amax = np.abs(g).max(-1)
    e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 8 + 127, 0)
    e = np.clip(e, 0, 254)
    codes = e4m3_codes(g / np.exp2(e - 127)[..., None])
    return codes.reshape(x.shape), np.where(bad, 255, e).astype(np.uint8)


def dequantise(codes, e):
    x = e4m3_values(codes).reshape(*e.shape, 32) * np.exp2(e.astype(np.float64) - 127)[..., None]
    return np.where((e == 255)[..., None], np.nan, x).reshape(codes.shape)


def rope_rows(x, pos, cos, sin):
    """fp32 rows [n, H, D] rotated at positions pos by fp32 tables, each operation rounded to fp32."""
    c, s = cos[pos][:, None, :].astype(np.float32), sin[pos][:, None, :].astype(np.float32)
    a, b = x[..., 0::2].astype(np.float32), x[..., 1::2].astype(np.float32)
    y = np.empty_like(x, dtype=np.float32)
    y[..., 0::2] = a * c - b * s
    y[..., 1::2] = a * s + b * c
    return y


def gather(pages, table, b, n):
    """Rows 0 .. n-1 of sequence b from float64 pages [n_pages, H, page, D]: [n, H, D]."""
    page = pages.shape[2]
    return np.stack([pages[table[b][p // page], :, p % page] for p in range(n)]) if n else \
        np.zeros((0, pages.shape[1], pages.shape[3]))


def activate(s, act):
    if act == "silu":
        return s / (1 + np.exp(-s))
    if act == "gelu":
        return 0.5 * s * (1 + np.tanh(math.sqrt(2 / math.pi) * (s + 0.044715 * s**3)))
    c, a = math.sqrt(2 / math.pi), 0.044715
    return s / 2 + c / 2 * s**2 + (c * a - c**3 / 3) / 2 * s**4 + (2 * c**5 / 15 - c**3 * a) / 2 * s**6


def allowed(lq, n, causal, window, block):
    """[lq, n] truth values by visiting every pair."""
    d = n - lq
    m = np.ones((lq, n), bool)
    for i in range(lq):
        for j in range(n):
            if causal or window:
                m[i, j] &= j <= i + d
            if window:
                m[i, j] &= i + d - j < window
            if block:
                m[i, j] &= j // block == (i + d) // block
    return m


def decode(q, k_pages, v_pages, table, kv_lens, q_off, act="softmax", causal=False, window=0, block=0, norm=False,
           scale=None, part=2.0**-16, floor=0.0):
    """q float64 [total, Hq, D]; pages float64. Returns o, lse and the elementwise bounds described in weights();
    ``part`` and ``floor``: how far a weight may be off as an operand of the second product, as a share of itself and of
    the row's largest."""
    total, Hq, D = q.shape
    H = k_pages.shape[1]
    G = Hq // H
    scale = D**-0.5 if not scale else scale
    o, lse = np.zeros_like(q), np.full((total, Hq), -np.inf)
    o_tol, lse_tol = np.zeros_like(q), np.zeros((total, Hq))
    for b, n in enumerate(kv_lens):
        lo, hi = q_off[b], q_off[b + 1]
        if hi <= lo:
            continue
        k, v = gather(k_pages, table, b, n), gather(v_pages, table, b, n)
        m = allowed(hi - lo, n, causal, window, block)
        for r in range(lo, hi):
            keep = m[r - lo]
            if not keep.any():
                continue
            for h in range(Hq):
                kk, vv = k[keep, h // G], v[keep, h // G]
                s = scale * (kk @ q[r, h])
                w, err = weights(s, scale * (np.abs(kk) @ np.abs(q[r, h])), act, len(s), part)
                if act == "softmax":
                    top = s.max()
                    lse[r, h] = top + np.log(np.exp(s - top).sum())
                    # each term is off by a factor within err; the logarithm's own and the final rounding
                    lse_tol[r, h] = err.max() + 2.0**-20 * (1 + abs(lse[r, h]))
                    w, err = np.exp(s - lse[r, h]), np.exp(s - lse[r, h]) * (err + err.max())
                err = err + floor * np.abs(w).max()
                c = 1.0 / n if norm else 1.0
                o[r, h] = c * (w @ vv)
                # rounding to bf16 (2^-8 relative) behind the sum's own error
                e = c * (err @ np.abs(vv))
                o_tol[r, h] = e + 2.0**-8 * (np.abs(o[r, h]) + e)
    return o, lse, o_tol, lse_tol


def weights(s, a, act, n, part):
    """(w, bound of its error): products of bf16 values are exact in fp32, so a score of D <= 128 terms summed in fp32
    is off by at most 2^-16 a, a = scale * sum |q_d k_d| (128 roundings of 2^-23). An exponential (or sigmoid) of it in
    fp32 adds its argument's rounding (2^-22 of |s| + 16, the running maximum's place) and 2^-20; weights enter the
    second product as two bf16 parts (2^-16) or, for an MXFP8 cache, rounded to fp16 (half a step: 2^-11), and are
    summed in fp32 (n roundings of 2^-23)."""
    rel = 2.0**-20 + 2.0**-22 * (np.abs(s) + 16) + part + n * 2.0**-23
    if act == "softmax":
        return None, rel + 2.0**-16 * a
    w = activate(s, act)
    # the activations' slopes stay below 1.2 (the polynomial's, on |s| <= 1.2, below 2)
    return w, np.abs(w) * rel + 2.0 * 2.0**-16 * a + 2.0**-20 * np.abs(s)
