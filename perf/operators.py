"""The paged key/value cache operators, measured: writing new rows into the
cache (bf16 or MXFP8 pages), reading rows back, and the attention of a few new
tokens per sequence over the cache.

``run`` computes them in their plain form with elementary torch operations in
32 bits (``own`` false) or makes the framework's calls (``own`` true); ``exact``
gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

SOFTMAX, SILU, GELU, GELU_POLY = "softmax", "silu", "gelu", "gelu_poly"


# ------------------------------------------------------------------ cases
def _decode(name, **kw):
    c = dict(name=name, op="decode", B=1, Hq=8, Hkv=8, D=128, page=64, fmt="bf16", lens="uniform", lo=1, hi=1000,
             max_lq=1, act=SOFTMAX, causal=False, window=0, block=0, norm=False)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(name=name, op="append", B=1, H=8, D=128, page=64, fmt="bf16", lens="uniform", lo=1, hi=1, cached=1000,
             rope=True)
    c.update(kw)
    return c


def _read(name, **kw):
    c = dict(name=name, op="read", B=1, H=8, D=128, page=64, fmt="bf16", lens="uniform", lo=1000, hi=1000, skip=0)
    c.update(kw)
    return c


def listed():
    return [
        # one user, one new event, a short history: latency is all there is
        _decode("decode_one_user", B=1, page=16, lo=777, hi=777),
        # a serving batch of the mixed workload's histories: most short, 30% between 4,000 and 32,000 events
        _decode("decode_mixed", B=64, lens="mixed", causal=True),
        # twice the users with the cache held in 8 bits
        _decode("decode_mixed_mxfp8", B=128, lens="mixed", fmt="mxfp8", causal=True),
        # four query heads share each key/value head; ordinary lengths, small pages
        _decode("decode_grouped", B=32, Hq=32, page=32, lo=1000, hi=8000),
        # up to eight candidate items scored at once against each history (pooling lengths), SiLU with the 1/L normaliser
        _decode("decode_candidates", B=64, lens="pma", max_lq=8, act=SILU, norm=True, fmt="mxfp8", page=128),
        # a single very long history, few key/value heads: the length has to be split
        _decode("decode_long", B=1, Hq=8, Hkv=2, D=64, lo=130001, hi=130001),
        # one event for each of 64 users, written to an 8-bit cache
        _append("append_events_mxfp8", B=64, fmt="mxfp8"),
        # whole histories (the jfa lengths) written once, keys rotated on the way
        _append("append_histories", B=128, H=4, lens="jfa", cached=0),
        # chunks of a few hundred rows appended behind what is cached, in 8 bits, keys as they come
        _append("append_chunks_mxfp8", B=256, lo=100, hi=900, cached=2000, fmt="mxfp8", rope=False, page=32),
        # one user's history read back for the jagged forward
        _read("read_one_user", lo=1001, hi=1001, page=16),
        # a batch of histories read back from 8 bits
        _read("read_histories_mxfp8", B=128, lens="jfa", fmt="mxfp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "read"])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["bf16", "mxfp8"])
    D = rng.choice([64, 128])
    B = _log(rng, 1, 300)
    if op == "decode":
        Hkv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 1, 2, 3, 4, 8])
        # at most 240,000 cached rows of 8 heads in all, at most 100,000 in one sequence
        hi = max(1, min(100000, 240000 * 8 // (B * Hkv)))
        hi = _log(rng, max(1, hi // 50), hi)
        act = rng.choice([SOFTMAX, SOFTMAX, SOFTMAX, SILU, GELU, GELU_POLY])
        mask = rng.choice(["none", "causal", "window", "block"])
        c = dict(op="decode", B=B, Hq=Hkv * group, Hkv=Hkv, D=D, page=page, fmt=fmt, lens="uniform",
                 lo=max(1, hi // rng.choice([1, 2, 10])), hi=hi, max_lq=rng.choice([1, 1, 2, 4, 7]), act=act,
                 causal=mask in ("causal", "window") or (mask == "block" and rng.random() < 0.5),
                 window=_log(rng, 16, 4000) if mask == "window" else 0,
                 block=_log(rng, 16, 4000) if mask == "block" else 0,
                 norm=act != SOFTMAX and rng.random() < 0.7)
        return c
    H = rng.choice([1, 2, 3, 4, 8])
    hi = _log(rng, 1, max(1, min(20000, 100000 * 8 // (B * H))))
    lo = max(1, hi // rng.choice([1, 2, 10]))
    if op == "append":
        return dict(op="append", B=B, H=H, D=D, page=page, fmt=fmt, lens="uniform", lo=lo, hi=hi,
                    cached=_log(rng, 1, 1000), rope=rng.random() < 0.6)
    return dict(op="read", B=B, H=H, D=D, page=page, fmt=fmt, lens="uniform", lo=lo, hi=hi,
                skip=rng.choice([0, 0, _log(rng, 1, 500)]))


def _lens(case, seed):
    """Rows per sequence (and what is cached before them): the length distributions of the repository's workloads.
    Every seed has the same lengths, so that outputs keep their shapes, in an order of its own."""
    order = np.random.default_rng(seed).permutation(case["B"])
    before = np.random.default_rng(1).integers(0, case.get("cached", 0) + 1, case["B"])
    return _drawn_lens(case)[order].astype(np.int64), before[order]


def _drawn_lens(case):
    rng = np.random.default_rng(0)
    B = case["B"]
    if case["lens"] == "mixed":
        n_long = int(round(0.3 * B))
        return rng.permutation(np.concatenate([rng.integers(50, 501, B - n_long), rng.integers(4000, 32001, n_long)]))
    if case["lens"] == "pma":
        return np.clip(np.rint(rng.lognormal(math.log(2048), 1.0, B)), 100, 20000).astype(np.int64)
    if case["lens"] == "jfa":
        return np.clip(np.rint(rng.lognormal(math.log(1024), 1.0, B)), 64, 16384).astype(np.int64)
    return rng.integers(case["lo"], case["hi"] + 1, B)


# ------------------------------------------------------------------ inputs
def _randn(shape, g, std=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return x if std == 1.0 else x * std


def _quantise(x):
    """x in 32 bits [..., D] to (E4M3 codes, E8M0 exponents [..., D/32]): one scale per 32 neighbours."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    field = g.abs().amax(-1).view(torch.int32) >> 23
    e = (field - 8).clamp(min=0)
    inv = ((254 - e) << 23).view(torch.float32)
    codes = (g * inv[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.reshape(x.shape), e.to(torch.uint8)


def _values(codes, scales, dtype):
    """The values that E4M3 codes (held as bytes) and E8M0 exponents stand for."""
    x = codes.view(torch.float8_e4m3fn).to(dtype).reshape(*scales.shape, 32)
    return (x * torch.exp2(scales.to(dtype) - 127.0)[..., None]).reshape(codes.shape)


def _pages(n_pages, H, page, D, fmt, g):
    """A cache's page buffers holding earlier rows: k, v (and their scales, or None)."""
    k, v = _randn((n_pages, H, page, D), g), _randn((n_pages, H, page, D), g)
    if fmt == "bf16":
        return k, v, None, None
    (kc, ks), (vc, vs) = _quantise(k.float()), _quantise(v.float())
    return kc.view(torch.uint8), vc.view(torch.uint8), ks, vs


def _table(lens, page, seed):
    """Page table int32 [B, max pages] with the pages in scattered order, and the number of pages."""
    need = -(-np.asarray(lens) // page)
    n = int(need.sum())
    ids = np.random.default_rng(seed + 1).permutation(n + 8)
    table = np.zeros((len(need), max(1, int(need.max()))), dtype=np.int32)
    first = np.cumsum(need) - need
    inside = np.arange(table.shape[1])[None, :] < need[:, None]
    table[inside] = ids[(first[:, None] + np.arange(table.shape[1])[None, :])[inside]]
    return torch.from_numpy(table).cuda(), n + 8


def _offsets(lens):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, page, D, B = case["op"], case["page"], case["D"], case["B"]
    lens, start = _lens(case, seed)
    s = dict(case=case)
    if op == "decode":
        s["table"], n = _table(lens, page, seed)
        s["k"], s["v"], s["ks"], s["vs"] = _pages(n, case["Hkv"], page, D, case["fmt"], g)
        lq = np.ones(B, np.int64) if case["max_lq"] == 1 else \
            np.random.default_rng(seed + 2).permutation(1 + np.arange(B) % case["max_lq"])
        # scores of pointwise activations stay where the polynomial holds
        s["q"] = _randn((int(lq.sum()), case["Hq"], D), g, 1.0 if case["act"] == SOFTMAX else 0.3)
        s["q_off"] = None if case["max_lq"] == 1 else _offsets(lq)
        s["kv_lens"] = torch.from_numpy(lens).cuda()
        return s
    if op == "append":
        s["table"], n = _table(lens + start, page, seed)
        s["k"], s["v"], s["ks"], s["vs"] = _pages(n, case["H"], page, D, case["fmt"], g)
        total = int(lens.sum())
        s["new_k"], s["new_v"] = _randn((total, case["H"], D), g), _randn((total, case["H"], D), g)
        s["start"] = torch.from_numpy(start).cuda()
        s["off"] = _offsets(lens)
        if case["rope"]:
            pos = torch.arange(int((lens + start).max()), device="cuda", dtype=torch.float64)
            theta = 10000.0 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
            angle = pos[:, None] * theta[None, :]
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        return s
    s["table"], n = _table(lens + case["skip"], page, seed)
    s["k"], s["v"], s["ks"], s["vs"] = _pages(n, case["H"], page, D, case["fmt"], g)
    s["off"], s["total"] = _offsets(lens), int(lens.sum())
    s["start"] = torch.full((B,), case["skip"], dtype=torch.int64, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"decode": _plain_decode, "append": _plain_append, "read": _plain_read}[s["case"]["op"]](s)


def _run_own(s):
    import jagged_attention_recsys_gdpa_gb300 as J

    c = s["case"]
    if "cache" not in s:  # the handle that a program makes once
        s["cache"] = J.PagedCache(s["k"], s["v"], s["ks"], s["vs"])
    cache = s["cache"]
    if c["op"] == "decode":
        o, lse = J.decode(s["q"], cache, s["table"], s["kv_lens"], q_off=s["q_off"], act=c["act"], causal=c["causal"],
                          window=c["window"], block=c["block"], norm_by_lkv=c["norm"])
        return dict(o=o) if lse is None else dict(o=o, lse=lse)
    if c["op"] == "append":
        J.cache_append(cache, s["new_k"], s["new_v"], s["table"], s["start"], off=s["off"],
                       rope=(s["cos"], s["sin"]) if c["rope"] else None)
        return _cache_out(s)
    k, v = J.cache_read(cache, s["table"], s["off"], start=s["start"], total=s["total"])
    return dict(k=k, v=v)


def _cache_out(s):
    """The cache as it stands: bf16 pages, or the codes' and the scales' values."""
    if s["ks"] is None:
        return dict(k=s["k"], v=s["v"])
    return dict(k=s["k"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn),
                ks=s["ks"].view(torch.float8_e8m0fnu), vs=s["vs"].view(torch.float8_e8m0fnu))


def _dense(pages, scales, table):
    """The cached rows of each sequence, in 32 bits: [B, H, max pages * page, D]."""
    x = pages[table].float() if scales is None else _values(pages[table], scales[table], torch.float32)
    B, P, H, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, P * page, D)


def _act(s, act):
    if act == SILU:
        return s / (1.0 + torch.exp(-s))
    if act == GELU:
        return 0.5 * s * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (s + 0.044715 * s * s * s)))
    c, a = math.sqrt(2.0 / math.pi), 0.044715
    s2 = s * s
    return 0.5 * s + s2 * (c / 2 + s2 * ((c * a - c**3 / 3) / 2 + s2 * ((2 * c**5 / 15 - c**3 * a) / 2)))


def _plain_decode(s):
    c, q = s["case"], s["q"].float()
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    G, LQ = Hq // Hkv, c["max_lq"]
    kv_len = s["kv_lens"]
    # the queries of each sequence, padded to LQ: q_pad [B, Hkv, G * LQ, D]
    if s["q_off"] is None:
        rows = torch.arange(B, device="cuda")[:, None]
        lq = torch.ones_like(kv_len)
    else:
        lq = s["q_off"][1:] - s["q_off"][:-1]
        rows = (s["q_off"][:-1, None] + torch.arange(LQ, device="cuda")[None, :]).clamp(max=q.shape[0] - 1)
    real = torch.arange(LQ, device="cuda")[None, :] < lq[:, None]
    q_pad = q[rows].reshape(B, LQ, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * LQ, D)
    k, v = _dense(s["k"], s["ks"], s["table"]), _dense(s["v"], s["vs"], s["table"])
    L = k.shape[2]
    score = (torch.matmul(q_pad, k.transpose(2, 3)) / math.sqrt(D)).reshape(B, Hkv, G, LQ, L)
    j = torch.arange(L, device="cuda")[None, None, :]
    p = (torch.arange(LQ, device="cuda")[None, :] + (kv_len - lq)[:, None])[:, :, None]  # position of each query
    keep = j < kv_len[:, None, None]
    if c["causal"] or c["window"]:
        keep = keep & (j <= p)
    if c["window"]:
        keep = keep & (j > p - c["window"])
    if c["block"]:
        keep = keep & (torch.div(j, c["block"], rounding_mode="floor") == torch.div(p, c["block"], rounding_mode="floor"))
    keep = keep.expand(B, LQ, L)[:, None, None]
    if c["act"] == SOFTMAX:
        score = score.masked_fill(~keep, -math.inf)
        top = score.amax(-1, keepdim=True)
        e = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        total = e.sum(-1, keepdim=True)
        w = e / torch.where(total > 0, total, torch.ones_like(total))
        lse = (top + torch.log(total))[..., 0]
    else:
        w, lse = torch.where(keep, _act(score, c["act"]), torch.zeros((), device="cuda")), None
        if c["norm"]:
            w = w / kv_len.clamp(min=1).float()[:, None, None, None, None]
    o = torch.matmul(w.reshape(B, Hkv, G * LQ, L), v).reshape(B, Hkv, G, LQ, D)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * LQ, Hq, D)
    # rows in the order of q: padded places dropped by a gather whose size q gives
    if s["q_off"] is not None:
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), lq, output_size=q.shape[0])
        at = b * LQ + torch.arange(q.shape[0], device="cuda") - s["q_off"][b]
        o = o[at]
        lse = None if lse is None else lse.permute(0, 3, 1, 2).reshape(B * LQ, Hq)[at]
    elif lse is not None:
        lse = lse.permute(0, 3, 1, 2).reshape(B, Hq)
    o = o.to(torch.bfloat16)
    return dict(o=o) if lse is None else dict(o=o, lse=lse)


def _row_places(s, total):
    """For each jagged row: its page, its place in the page and its position."""
    page = s["case"]["page"]
    b = torch.repeat_interleave(torch.arange(s["case"]["B"], device="cuda"), s["off"][1:] - s["off"][:-1],
                                output_size=total)
    pos = s["start"][b] + torch.arange(total, device="cuda") - s["off"][b]
    return s["table"][b, pos // page].long(), pos % page, pos


def _plain_append(s):
    pg, at, pos = _row_places(s, s["new_k"].shape[0])
    k, v = s["new_k"].float(), s["new_v"].float()
    if s["case"]["rope"]:
        cos, sin = s["cos"][pos][:, None, :], s["sin"][pos][:, None, :]
        x, y = k[..., 0::2], k[..., 1::2]
        k = torch.stack([x * cos - y * sin, x * sin + y * cos], dim=-1).reshape(k.shape)
    if s["ks"] is None:
        s["k"][pg, :, at] = k.to(torch.bfloat16)
        s["v"][pg, :, at] = v.to(torch.bfloat16)
        return _cache_out(s)
    new_k, new_v = _quantise(k), _quantise(v)
    s["k"][pg, :, at], s["ks"][pg, :, at] = new_k[0].view(torch.uint8), new_k[1]
    s["v"][pg, :, at], s["vs"][pg, :, at] = new_v[0].view(torch.uint8), new_v[1]
    return _cache_out(s)


def _plain_read(s):
    pg, at, _ = _row_places(s, s["total"])
    k, v = s["k"][pg, :, at], s["v"][pg, :, at]
    if s["ks"] is None:
        return dict(k=k, v=v)
    return dict(k=_values(k, s["ks"][pg, :, at], torch.float32).to(torch.bfloat16),
                v=_values(v, s["vs"][pg, :, at], torch.float32).to(torch.bfloat16))


# ------------------------------------------------------------------ work
def work(case):
    D, page, B = case["D"], case["page"], case["B"]
    elt = 2 * D if case["fmt"] == "bf16" else D + D // 32  # bytes of one cached row of one head
    n = _drawn_lens(case).astype(np.float64)
    if case["op"] == "decode":
        lq = 1 + np.arange(B) % case["max_lq"]
        seen = n  # keys that some query of the sequence sees
        if case["window"]:
            seen = np.minimum(n, case["window"] + lq - 1)
        if case["block"]:  # the blocks of the sequence's last lq positions
            seen = np.minimum(n, n - np.floor((n - lq) / case["block"]) * case["block"])
        rows = float(lq.sum())
        cache = float(seen.sum()) * case["Hkv"] * 2 * elt
        q = rows * case["Hq"] * (4 * D + (4 if case["act"] == SOFTMAX else 0))
        return dict(bytes=cache + q + 8 * B + 4 * float(np.ceil(seen / page).sum()),
                    flops=4 * D * case["Hq"] * float((lq * seen).sum()))
    rows, H = float(n.sum()), case["H"]
    moved = rows * H * 2 * (2 * D + elt)
    if case["op"] == "append":
        rope = rows * 4 * D if case["rope"] else 0  # a row's cos and sin
        return dict(bytes=moved + rope, flops=rows * H * D * (3 if case["rope"] else 1))
    return dict(bytes=moved, flops=rows * H * D)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    table = s["table"].long().cpu()
    page, D = case["page"], case["D"]
    if case["op"] == "decode":
        lens = s["kv_lens"].tolist()
        starts = list(range(case["B"] + 1)) if s["q_off"] is None else s["q_off"].tolist()
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        G = case["Hq"] // case["Hkv"]
        for b, n in enumerate(lens):
            first, nq = starts[b], starts[b + 1] - starts[b]
            k, v = (_sequence(s[x], s[x + "s"], table[b], n, page) for x in ("k", "v"))
            i, j = torch.arange(nq, device="cuda")[:, None] + (n - nq), torch.arange(n, device="cuda")[None, :]
            seen = torch.ones(nq, n, dtype=torch.bool, device="cuda")
            if case["causal"] or case["window"]:
                seen &= j <= i
            if case["window"]:
                seen &= i - j < case["window"]
            if case["block"]:
                w = case["block"]
                seen &= torch.floor(j.double() / w) == torch.floor(i.double() / w)
            for h in range(case["Hkv"]):
                heads = slice(h * G, (h + 1) * G)
                z = torch.einsum("qgd,nd->qgn", s["q"][first:first + nq, heads].double(), k[h]) * D**-0.5
                m = seen[:, None, :]
                if case["act"] == SOFTMAX:
                    z = z.masked_fill(~m, -math.inf)
                    lse[first:first + nq, heads] = torch.logsumexp(z, -1)
                    w8 = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
                else:
                    if case["act"] == SILU:
                        w8 = z * torch.sigmoid(z)
                    elif case["act"] == GELU:
                        w8 = 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z**3)))
                    else:
                        r = (2 / math.pi) ** 0.5
                        w8 = z / 2 + r / 2 * z**2 + (r * 0.044715 - r**3 / 3) / 2 * z**4 \
                            + (2 * r**5 / 15 - r**3 * 0.044715) / 2 * z**6
                    w8 = w8 * m / (n if case["norm"] else 1)
                o[first:first + nq, heads] = torch.einsum("qgn,nd->qgd", w8, v[h])
        return dict(o=o) if case["act"] != SOFTMAX else dict(o=o, lse=lse)
    lens = (s["off"][1:] - s["off"][:-1]).tolist()
    start = s["start"].tolist()
    if case["op"] == "read":
        k, v = (torch.cat([_sequence(s[x], s[x + "s"], table[b], start[b] + n, page)[:, start[b]:]
                           for b, n in enumerate(lens)], dim=1).transpose(0, 1) for x in ("k", "v"))
        return dict(k=k.contiguous(), v=v.contiguous())
    # append: the rows in 64 bits, laid into the cache as it was
    pos = torch.cat([torch.arange(p, p + n) for p, n in zip(start, lens)]).cuda()
    which = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)])
    pages = table[which, pos.cpu() // page].cuda()
    k, v = s["new_k"].double(), s["new_v"].double()
    if case["rope"]:
        turn = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None, :]
        k = torch.view_as_real(torch.view_as_complex(k.reshape(*k.shape[:-1], D // 2, 2)) * turn).reshape(k.shape)
    out = {}
    for name, new in (("k", k), ("v", v)):
        if s[name + "s"] is None:
            whole = s[name].double()
            whole[pages, :, pos % page] = new
            out[name] = whole
            continue
        values = s[name].view(torch.float8_e4m3fn).double()
        scale = torch.exp2(s[name + "s"].double() - 127)
        blocks = new.reshape(*new.shape[:-1], D // 32, 32)
        top = blocks.abs().amax(-1)
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(top.clamp(min=1e-300))) - 8, min=-127))
        values[pages, :, pos % page] = _nearest_e4m3(blocks / step[..., None]).reshape(new.shape)
        scale[pages, :, pos % page] = step
        out[name], out[name + "s"] = values, scale
    return out


def _sequence(pages, scales, ids, n, page):
    """Cached rows 0 .. n-1 of one sequence in 64 bits: [H, n, D]."""
    ids = ids[: -(-n // page)].cuda()
    x = pages[ids]
    if scales is None:
        x = x.double()
    else:
        x = _values(x, scales[ids], torch.float64)
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n]


def _nearest_e4m3(x):
    """The E4M3 value nearest to x (ties to even), saturated at 448, in 64 bits."""
    a = x.abs().clamp(max=448.0)
    ulp = torch.exp2(torch.clamp(torch.floor(torch.log2(a.clamp(min=1e-300))), min=-6) - 3)
    return torch.sign(x) * torch.round(a / ulp) * ulp
