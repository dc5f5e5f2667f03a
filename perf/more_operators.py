"""What stands between a model's projections and jagged attention, measured:
layer norm of rows (forward, and backward with the weight's and the bias'
gradients), rotary positions in either layout, the cos / sin tables of far
positions, and page tables with slots made on the GPU from request lengths.

``run`` computes them in their plain form with elementary torch operations in
32 bits, angles in 64 (``own`` false), or makes the framework's calls (``own``
true); ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _norm(name, **kw):
    # x [rows, heads, N]; beside: more heads of the same fused tensor behind them; pad: rows behind the last sequence
    c = dict(name=name, op="norm", back=False, rows=1, heads=1, N=128, type="bf16", weight="fp32", beside=0, pad=0)
    c.update(kw)
    return c


def _rotary(name, **kw):
    # lens "rows": every row stands at a position of its own (B rows)
    c = dict(name=name, op="rotary", B=1, lens="uniform", lo=1, hi=1, heads=8, D=128, R=128, layout="interleaved",
             inverse=False, type="bf16", beside=0, start=0)
    c.update(kw)
    return c


def _tables(name, **kw):
    c = dict(name=name, op="tables", rows=4096, dim=64, base=10000.0, scaling="none", factor=1.0, original=4096)
    c.update(kw)
    return c


def _pages(name, **kw):
    c = dict(name=name, op="pages", B=1, lens="uniform", lo=1, hi=1, kept=0, page=64, spare=64)
    c.update(kw)
    return c


def listed():
    return [
        # a serving step: the query and key heads of 64 new events, inside the fused projection's rows
        _norm("norm_tokens", rows=64, heads=10, beside=2),
        # query rows of a training batch of histories (the jfa lengths), a row per head
        _norm("norm_histories", rows=212788, heads=4),
        # events at model width, of a size that no vector divides
        _norm("norm_odd_width", rows=30011, N=1001, type="fp16", weight="fp16"),
        # the histories' backward pass, its weight's gradient summed over 851,152 rows
        _norm("norm_back_histories", rows=212788, heads=4, back=True),
        # model-width rows held in 32 bits, a padded batch
        _norm("norm_back_wide", rows=8000, N=4096, type="fp32", back=True, pad=77),
        # a serving step: 64 events at their own positions, query and key heads of the fused projection
        _rotary("rotary_tokens", B=64, lens="rows", hi=32000, heads=10, beside=2, layout="half"),
        # query and key heads of a training batch of histories together
        _rotary("rotary_histories", B=128, lens="jfa", heads=8),
        # gradients rotated back, half of each head's columns, three heads, chunks behind earlier rows
        _rotary("rotary_back_part", B=256, lo=100, hi=900, heads=3, R=64, layout="half", inverse=True, type="fp16",
                start=2000),
        # tables made anew as a user's context grows
        _tables("tables_short", rows=4096, dim=64, scaling="ntk", factor=2.0),
        # tables of a long context, sixteen times what the model was trained on
        _tables("tables_long", rows=262144, dim=128, scaling="yarn", factor=16.0, original=16384),
        # a serving step of 64 users: one event each, taken back and placed again
        _pages("pages_tokens", B=64, kept=32000),
        # the mixed workload's batch leaves and the next one comes
        _pages("pages_histories", B=1024, lens="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "rotary", "rotary", "tables", "pages"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "norm":
        N = rng.choice([64, 128, 128, _log(rng, 16, 8192), 8 * _log(rng, 2, 1024)])
        heads = rng.choice([1, 1, 2, 4, 5, 8]) if N <= 256 else 1
        most = 100_000_000 if kind != "fp32" else 50_000_000
        return dict(op="norm", back=rng.random() < 0.5, rows=_log(rng, 1, min(200_000, most // (N * heads))),
                    heads=heads, N=N, type=kind, weight=rng.choice(["fp32", kind, "none"]),
                    beside=rng.choice([0, 0, 1, 2]), pad=rng.choice([0, 0, 0, 5]))
    if op == "rotary":
        D = rng.choice([64, 128, 128, 32, 80, 96, 2 * _log(rng, 1, 128)])
        heads = rng.choice([1, 2, 3, 4, 8, 10, 16])
        B = _log(rng, 1, 300)
        hi = _log(rng, 1, max(1, min(20000, 100_000_000 // (2 * B * heads * D))))
        rows = rng.random() < 0.3
        return dict(op="rotary", B=_log(rng, 1, 2000) if rows else B, lens="rows" if rows else "uniform",
                    lo=max(1, hi // rng.choice([1, 2, 10])), hi=hi, heads=heads, D=D,
                    R=max(2, D // rng.choice([1, 1, 2, 4]) // 2 * 2), layout=rng.choice(["interleaved", "half"]),
                    inverse=rng.random() < 0.4, type=kind, beside=rng.choice([0, 0, 1, 2]),
                    start=rng.choice([0, 0, 1000]))
    if op == "tables":
        dim = rng.choice([64, 128, 2 * _log(rng, 1, 128)])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"]) if dim > 2 else rng.choice(["none", "linear", "yarn"])
        return dict(op="tables", rows=_log(rng, 1, 30_000_000 // max(128, dim)), dim=dim,
                    base=rng.choice([10000.0, 500000.0]), scaling=scaling, original=rng.choice([2048, 4096, 16384]),
                    factor=1.0 if scaling == "none" else rng.choice([1.5, 2.0, 8.0, 32.0]))
    B = _log(rng, 1, 2000)
    hi = rng.choice([1, 1, 8, _log(rng, 1, 4_000_000 // B)])
    return dict(op="pages", B=B, lens="uniform", lo=max(1, hi // rng.choice([1, 2, 10])), hi=hi,
                kept=rng.choice([0, _log(rng, 1, 4_000_000 // B)]), page=rng.choice([8, 16, 32, 64, 128, 256]),
                spare=rng.choice([0, 100]))


def _lens(case):
    """New rows of each sequence and the rows before them: the length distributions of the repository's workloads, the
    same for every seed, so that outputs keep their shapes."""
    rng = np.random.default_rng(0)
    B = case["B"]
    before = np.random.default_rng(1).integers(0, case.get("kept", case.get("start", 0)) + 1, B)
    if case["lens"] == "mixed":
        n_long = int(round(0.3 * B))
        n = rng.permutation(np.concatenate([rng.integers(50, 501, B - n_long), rng.integers(4000, 32001, n_long)]))
    elif case["lens"] == "jfa":
        n = np.clip(np.rint(rng.lognormal(math.log(1024), 1.0, B)), 64, 16384)
    elif case["lens"] == "rows":
        n = np.ones(B)
    else:
        n = rng.integers(case["lo"], case["hi"] + 1, B)
    return n.astype(np.int64), before.astype(np.int64)


# ------------------------------------------------------------------ inputs
def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _offsets(lens):
    return _cuda(np.concatenate([[0], np.cumsum(lens)]).astype(np.int64))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        return _prepare_norm(s, case, g)
    if case["op"] == "rotary":
        return _prepare_rotary(s, case, g, seed)
    if case["op"] == "tables":
        # nothing but numbers: another seed is another base
        s["base"] = case["base"] * (1.0 + (seed % 997) / 1000.0)
        return s
    return _prepare_pages(s, case, seed)


def _prepare_norm(s, c, g):
    rows, heads, N, kind = c["rows"] + c["pad"], c["heads"], c["N"], TYPES[c["type"]]

    def activations(std):
        return torch.randn((rows, heads + c["beside"], N), generator=g, device="cuda", dtype=kind) * std

    # projections' outputs: not centred, of a size of their own in each column, a few columns far larger
    column = torch.exp(torch.randn(N, generator=g, device="cuda") * 0.3)
    column = torch.where(torch.rand(N, generator=g, device="cuda") < 0.02, column * 8.0, column)
    shift = torch.randn(N, generator=g, device="cuda") * 0.5
    x = activations(1.0)
    x.mul_(column.to(kind)).add_(shift.to(kind))
    s["x"] = x[:, :heads]
    if c["weight"] == "none":
        s["w"] = s["b"] = None
    else:
        w = TYPES[c["weight"]]
        s["w"] = (1.0 + 0.1 * torch.randn(N, generator=g, device="cuda")).to(w)
        s["b"] = (0.1 * torch.randn(N, generator=g, device="cuda")).to(w)
    s["off"] = _cuda(np.array([0, c["rows"] // 2, c["rows"]])) if c["pad"] else None
    if c["back"]:
        s["dy"] = activations(0.1)[:, :heads]
        wide = s["x"].double()
        mean = wide.mean(-1)
        s["mean"] = mean.float()
        s["rstd"] = ((wide - mean[..., None]).square().mean(-1) + EPS).rsqrt().float()
    return s


def _prepare_rotary(s, c, g, seed):
    lens, before = _lens(c)
    total = int(lens.sum())
    x = torch.randn((total, c["heads"] + c["beside"], c["D"]), generator=g, device="cuda", dtype=TYPES[c["type"]])
    s["x"] = x[:, :c["heads"]]
    if c["lens"] == "rows":
        s["off"], s["start"] = None, _cuda(np.random.default_rng(seed).integers(0, c["hi"], c["B"]))
        longest = c["hi"]
    else:
        order = np.random.default_rng(seed).permutation(c["B"])
        lens, before = lens[order], before[order]
        s["off"], s["start"] = _offsets(lens), _cuda(before) if c["start"] else None
        longest = int((lens + before).max())
    turn = torch.arange(longest, device="cuda", dtype=torch.float64)[:, None] * _theta(c["R"], 10000.0)[None, :]
    s["cos"], s["sin"] = turn.cos().float(), turn.sin().float()
    return s


def _prepare_pages(s, c, seed):
    lens, before = _lens(c)
    order = np.random.default_rng(seed).permutation(c["B"])
    lens, before = lens[order], before[order]
    # earlier rows hold whole pages in part, so a new row may need no page
    need = -(-(lens + before) // c["page"])
    n = int(need.sum()) + c["spare"]
    ids = np.random.default_rng(seed + 1).permutation(n).astype(np.int32)
    table = np.full((c["B"], int(need.max()) + 3), -1, np.int32)
    inside = np.arange(table.shape[1])[None, :] < need[:, None]
    table[inside] = ids[:int(need.sum())]
    free = np.full(n, -1, np.int32)
    free[:c["spare"]] = ids[int(need.sum()):]
    s.update(table=_cuda(table), free=_cuda(free), count=_cuda(np.array([c["spare"]])), off=_offsets(lens),
             start=_cuda(before), lens=_cuda(lens + before), total=int(lens.sum()))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_norm, "rotary": _plain_rotary, "tables": _plain_tables, "pages": _plain_pages}[s["case"]["op"]](s)


def _run_own(s):
    import jagged_attention_recsys_gdpa_gb300 as J

    c = s["case"]
    if c["op"] == "norm":
        if c["back"]:
            dx, dw, db = J.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], off=s["off"])
            return dict(dx=dx) if s["w"] is None else dict(dx=dx, dw=dw, db=db)
        y, mean, rstd = J.layer_norm_forward(s["x"], s["w"], s["b"], eps=EPS, off=s["off"])
        return dict(y=y, mean=mean, rstd=rstd)
    if c["op"] == "rotary":
        return dict(y=J.rotary(s["x"], (s["cos"], s["sin"]), off=s["off"], start=s["start"], layout=c["layout"],
                               inverse=c["inverse"]))
    if c["op"] == "tables":
        cos, sin = J.rotary_tables(c["rows"], c["dim"], base=s["base"], scaling=c["scaling"], factor=c["factor"],
                                   original=c["original"])
        return dict(cos=cos, sin=sin)
    if "pool" not in s:  # the handle that a program makes once
        s["pool"] = J.PagePool(s["free"], s["count"], c["page"])
    J.page_release(s["pool"], s["table"], s["lens"], keep=s["start"])
    slots = J.page_assign(s["pool"], s["table"], s["start"], off=s["off"], total=s["total"])
    return dict(slots=slots, table=s["table"], free=s["free"], count=s["count"])


def _live(s, x):
    """x with zeros in the rows behind the last sequence."""
    if s["off"] is None:
        return x
    real = torch.arange(x.shape[0], device="cuda") < s["off"][-1]
    return torch.where(real.reshape(-1, *[1] * (x.dim() - 1)), x, torch.zeros((), dtype=x.dtype, device="cuda"))


def _plain_norm(s):
    x, kind, N = s["x"].float(), s["x"].dtype, s["x"].shape[-1]
    if not s["case"]["back"]:
        mean = x.sum(-1) / N
        d = x - mean[..., None]
        rstd = 1.0 / torch.sqrt((d * d).sum(-1) / N + EPS)
        y = d * rstd[..., None]
        if s["w"] is not None:
            y = y * s["w"].float() + s["b"].float()
        return dict(y=_live(s, y.to(kind)), mean=_live(s, mean), rstd=_live(s, rstd))
    dy = s["dy"].float()
    h = (x - s["mean"][..., None]) * s["rstd"][..., None]
    g = dy if s["w"] is None else dy * s["w"].float()
    dx = s["rstd"][..., None] * (g - g.sum(-1, keepdim=True) / N - h * ((g * h).sum(-1, keepdim=True) / N))
    if s["w"] is None:
        return dict(dx=_live(s, dx.to(kind)))
    return dict(dx=_live(s, dx.to(kind)), dw=_live(s, dy * h).sum((0, 1)).to(s["w"].dtype),
                db=_live(s, dy).sum((0, 1)).to(s["w"].dtype))


def _positions(s, total):
    """Each row's sequence and position."""
    if s["off"] is None:
        return None, s["start"]
    b = torch.repeat_interleave(torch.arange(s["case"]["B"], device="cuda"), s["off"][1:] - s["off"][:-1],
                                output_size=total)
    pos = torch.arange(total, device="cuda") - s["off"][b]
    return b, pos if s["start"] is None else pos + s["start"][b]


def _plain_rotary(s):
    c, x = s["case"], s["x"].float()
    half = c["R"] // 2
    _, pos = _positions(s, x.shape[0])
    cos, sin = s["cos"][pos][:, None, :], s["sin"][pos][:, None, :]
    if c["inverse"]:
        sin = -sin
    if c["layout"] == "half":
        a, b = x[..., :half], x[..., half:c["R"]]
    else:
        a, b = x[..., 0:c["R"]:2], x[..., 1:c["R"]:2]
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([u, v], -1) if c["layout"] == "half" else torch.stack([u, v], -1).reshape(*x.shape[:2], c["R"])
    return dict(y=torch.cat([turned, x[..., c["R"]:]], -1).to(s["x"].dtype))


def _theta(dim, base, scaling="none", factor=1.0, original=4096):
    """Angles per position of the dim / 2 pairs, in 64 bits."""
    m = torch.arange(dim // 2, device="cuda", dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    theta = base ** (-2.0 * m / dim)
    if scaling == "linear":
        theta = theta / factor
    if scaling == "yarn":  # pairs that turn often within the original length stay, slow ones are interpolated
        turns = original * theta / (2.0 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        theta = theta / factor * (1.0 - keep) + theta * keep
    return theta


def _plain_tables(s):
    c = s["case"]
    theta = _theta(c["dim"], s["base"], c["scaling"], c["factor"], c["original"])
    turn = torch.arange(c["rows"], device="cuda", dtype=torch.float64)[:, None] * theta[None, :]
    size = 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0
    return dict(cos=(turn.cos() * size).float(), sin=(turn.sin() * size).float())


def _plain_pages(s):
    table, free, page = s["table"], s["free"], s["case"]["page"]
    B, P = table.shape
    n, j = free.numel(), torch.arange(P, device="cuda")[None, :]
    low, high = (s["start"] + page - 1) // page, (s["lens"] + page - 1) // page
    first = torch.cumsum(high - low, 0) - (high - low)
    wanted, moved = first + high - low, (j >= low[:, None]) & (j < high[:, None])
    i = first[:, None] + j - low[:, None]  # its number among the pages that move
    # given back: the last of them at the bottom, so that the first is taken next; one place more for those that stay
    at = torch.where(moved, s["count"] + wanted[-1] - 1 - i, torch.full_like(i, n))
    stack = torch.cat([free, free.new_zeros(1)]).scatter_(0, at.reshape(-1), table.reshape(-1))[:n]
    count = s["count"] + wanted[-1]
    free.copy_(stack)
    table.copy_(torch.where(moved, torch.full_like(table, -1), table))
    # taken again
    at = torch.where(moved, count - 1 - i, torch.zeros_like(i))
    table.copy_(torch.where(moved, free[at], table))
    s["count"].copy_(count - wanted[-1])
    b, pos = _positions(s, s["total"])
    slots = table[b, pos // page].long() * page + pos % page
    return dict(slots=slots, table=table, free=free, count=s["count"])


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "norm":
        rows, N = case["rows"] * case["heads"], case["N"]
        size = TYPES[case["type"]].itemsize
        weights = 0 if case["weight"] == "none" else 2 * N * TYPES[case["weight"]].itemsize
        if case["back"]:
            return dict(bytes=rows * (3 * N * size + 8) + 1.5 * weights, flops=14 * rows * N)
        return dict(bytes=rows * (2 * N * size + 8) + weights, flops=8 * rows * N)
    if case["op"] == "rotary":
        lens, before = _lens(case)
        rows, half = int(lens.sum()), case["R"] // 2
        positions = min(case["hi"], case["B"]) if case["lens"] == "rows" else int((lens + before).max())
        return dict(bytes=2 * rows * case["heads"] * case["D"] * TYPES[case["type"]].itemsize + 8 * positions * half + 8 * case["B"],
                    flops=6 * rows * case["heads"] * half)
    if case["op"] == "tables":
        return dict(bytes=4 * case["rows"] * case["dim"], flops=case["rows"] * case["dim"] * 10)
    lens, before = _lens(case)
    moved = int((-(-(lens + before) // case["page"]) + -before // case["page"]).sum())
    # a page moves from the table to the pool and back, each time read and written; a row gets its slot
    return dict(bytes=16 * moved + 8 * int(lens.sum()) + 24 * case["B"], flops=int(lens.sum()))


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotary": _exact_rotary, "tables": _exact_tables, "pages": _exact_pages}[case["op"]](case, s)


def _exact_norm(c, s):
    out = {}
    n = c["rows"]
    x = s["x"].double()
    w = None if s["w"] is None else s["w"].double()
    mean = x.mean(-1, keepdim=True)
    scale = 1.0 / torch.sqrt(x.var(-1, unbiased=False, keepdim=True) + EPS)
    if not c["back"]:
        y = (x - mean) * scale
        out["y"] = y if w is None else torch.addcmul(s["b"].double(), y, w)
        out["mean"], out["rstd"] = mean[..., 0], scale[..., 0]
        for v in out.values():
            v[n:] = 0
        return out
    # the gradient of sum(dy * y): the Jacobian of a normalised row is (I - 1 1'/N - h h'/N) / sigma
    mean, scale = s["mean"].double()[..., None], s["rstd"].double()[..., None]
    h = (x - mean).mul_(scale)
    dy = s["dy"].double()
    g = dy if w is None else dy * w
    out["dx"] = (g - g.mean(-1, keepdim=True) - h * torch.einsum("rhn,rhn->rh", g, h)[..., None] / c["N"]) * scale
    out["dx"][n:] = 0
    if w is not None:
        out["dw"] = torch.einsum("rhn,rhn->n", dy[:n], h[:n])
        out["db"] = torch.einsum("rhn->n", dy[:n])
    return out


def _exact_rotary(c, s):
    x = s["x"].double()
    half, total = c["R"] // 2, x.shape[0]
    if s["off"] is None:
        pos = s["start"]
    else:
        ends = s["off"].tolist()
        first = [0] * c["B"] if s["start"] is None else s["start"].tolist()
        pos = torch.cat([torch.arange(p, p + ends[b + 1] - ends[b]) for b, p in enumerate(first)]).cuda()
    turn = torch.complex(s["cos"].double(), s["sin"].double())[pos].reshape(total, 1, half)
    if c["inverse"]:
        turn = turn.conj()
    y = x.clone()
    if c["layout"] == "half":
        z = torch.complex(x[..., :half].contiguous(), x[..., half:c["R"]].contiguous()) * turn
        y[..., :half], y[..., half:c["R"]] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:c["R"]:2].contiguous(), x[..., 1:c["R"]:2].contiguous()) * turn
        y[..., 0:c["R"]:2], y[..., 1:c["R"]:2] = z.real, z.imag
    return dict(y=y)


def _exact_tables(c, s):
    size, factor, theta = 1.0, c["factor"], []
    for m in range(c["dim"] // 2):
        base = s["base"] * factor ** (c["dim"] / (c["dim"] - 2.0)) if c["scaling"] == "ntk" else s["base"]
        t = math.exp(-math.log(base) * 2 * m / c["dim"])
        if c["scaling"] == "linear":
            t /= factor
        if c["scaling"] == "yarn":
            r = c["original"] * t / (2 * math.pi)
            part = min(1.0, max(0.0, (r - 1.0) / 31.0))
            t = (1.0 - part) * t / factor + part * t
            size = 0.1 * math.log(factor) + 1.0
        theta.append(t)
    turns = torch.arange(c["rows"], device="cuda", dtype=torch.float64)[:, None] \
        * (torch.tensor(theta, device="cuda", dtype=torch.float64) / (2 * math.pi))
    z = torch.polar(torch.full_like(turns, size), 2 * math.pi * (turns - torch.round(turns)))
    return dict(cos=z.real.contiguous(), sin=z.imag.contiguous())


def _exact_pages(c, s):
    """The pool as a list, one page after another."""
    page = c["page"]
    table, free, lens, start, off = (s[k].cpu().numpy() for k in ("table", "free", "lens", "start", "off"))
    pool = free[:int(s["count"].item())].tolist()
    back = []
    span = [(-(-int(a) // page), -(-int(z) // page)) for a, z in zip(start, lens)]
    for b, (lo, hi) in enumerate(span):
        back += table[b, lo:hi].tolist()
        table[b, lo:hi] = -1
    pool += back[::-1]
    stack = free.copy()
    stack[:len(pool)] = pool
    slots = np.zeros(int(off[-1]), np.int64)
    for b, (lo, hi) in enumerate(span):
        for j in range(lo, hi):
            table[b, j] = pool.pop()
        at = np.arange(start[b], lens[b])
        slots[off[b]:off[b + 1]] = table[b, at // page].astype(np.int64) * page + at % page
    return dict(slots=slots, table=table, free=stack, count=np.array([len(pool)]))
