"""The paged key/value cache on the GPU: appending (bf16 and MXFP8, rotated
keys), reading back, and the attention of new rows over it, against the plain
64-bit reference in paged_ref."""
import numpy as np
import pytest
import torch

from jagged_attention_recsys_gdpa_gb300 import inputs
from tests import paged_ref as R
from tests.dense_ref import rope_tables

pytestmark = pytest.mark.gpu

OFFSETS, ROPE, PAGES, LENGTH = 5, 9, 10, 11


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make_table(lens, page, seed, spare=3, extra_cols=0):
    """Scattered pages for sequences of the given lengths; unused entries hold no page at all."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // page) for n in lens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(1, max(need)) + extra_cols), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(need) + spare


def fill_cache(J, lens, page, H, D, fmt, seed, garbage=True, extra_cols=0, std=1.0):
    """A cache whose sequences hold random rows; every other place of its pages holds NaN. Returns the cache, the
    table and the float64 pages."""
    table, n_pages = make_table(lens, page, seed, extra_cols=extra_cols)
    rng = np.random.default_rng(seed + 1)
    live = np.zeros((n_pages, page), bool)
    for b, n in enumerate(lens):
        for p in range(int(n)):
            live[table[b, p // page], p % page] = True
    bufs, pages = [], []
    for _ in range(2):
        x = torch.from_numpy(rng.standard_normal((n_pages, H, page, D)) * std).to(torch.bfloat16)
        if fmt == "bf16":
            y = np64(x)
            if garbage:
                x[torch.from_numpy(~live)[:, None, :].expand(n_pages, H, page)] = float("nan")
            bufs.append((x.cuda(), None))
        else:
            codes, e = R.quantise(np64(x))
            y = R.dequantise(codes, e)
            if garbage:
                dead = np.broadcast_to(~live[:, None, :], (n_pages, H, page))
                codes = codes.copy()
                codes[dead], e[dead] = 0x7f, 255
            bufs.append((torch.from_numpy(codes).cuda(), torch.from_numpy(e).cuda()))
        pages.append(y)
    cache = J.PagedCache(bufs[0][0], bufs[1][0], bufs[0][1], bufs[1][1])
    return cache, table, pages


def prefix(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def clear(J):
    J.device_status()
    J.device_status()


# ------------------------------------------------------------------ append and read
def snapshot(cache):
    return [None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]


def expect_append(before, table, page, start, off, k, v, fmt, cos=None, sin=None):
    """The buffers after appending, from the definition (numpy, on the snapshot)."""
    want = [None if t is None else t.cpu().clone() for t in before]
    for b in range(len(start)):
        if start[b] < 0:
            continue
        for r in range(off[b], off[b + 1]):
            pos = start[b] + r - off[b]
            pg, at = table[b, pos // page], pos % page
            kr = k[r:r + 1].float().numpy()
            if cos is not None:
                kr = R.rope_rows(kr, np.array([pos]), cos, sin)
            for x, i in ((kr[0], 0), (v[r].float().numpy(), 1)):
                if fmt == "bf16":
                    want[i][pg, :, at] = torch.from_numpy(x).to(torch.bfloat16)
                else:
                    codes, e = R.quantise(x.astype(np.float64))
                    codes = np.where(np.repeat(e == 255, 32, axis=-1), 0, codes)
                    want[i][pg, :, at] = torch.from_numpy(codes)
                    want[2 + i][pg, :, at] = torch.from_numpy(e)
    return want


def same_bits(got, want):
    for g, w in zip(got, want):
        if w is not None:
            g, w = g.cpu().contiguous(), w.contiguous()
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("rope", [False, True], ids=["plain", "rope"])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("D,page,H", [(128, 16, 3), (64, 8, 1), (64, 64, 2), (128, 4096, 1)])
def test_append_writes_the_rows_and_nothing_else(D, page, H, fmt, rope):
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    new = [5, 0, 1, 33, 2]
    start = np.array([0, 9, 15, 30, -1])
    off = prefix(new)
    table, n_pages = make_table(np.array(new) + np.maximum(start, 0), page, seed=3)
    cache = J.paged_cache(n_pages, page, H, D, fmt)
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        if t is not None:
            t.view(torch.uint8).random_(0, 120)
    before = snapshot(cache)
    g = torch.Generator().manual_seed(4)
    total = int(off[-1]) + 3  # rows behind the last sequence
    k, v = (torch.randn(total, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    cos, sin, _ = rope_tables(128, D)
    cos, sin = cos.astype(np.float32), sin.astype(np.float32)
    J.cache_append(cache, k.cuda(), v.cuda(), cu(table), cu(start), off=cu(off), rope=(cu(cos), cu(sin)) if rope else None)
    assert J.device_status() == 0
    same_bits(snapshot(cache), expect_append(before, table, page, start, off, k, v, fmt, *((cos, sin) if rope else ())))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_append_one_row_per_sequence(fmt):
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    B, H, D, page = 37, 4, 128, 32
    start = np.random.default_rng(0).integers(0, 100, B)
    start[5] = -1  # a padded place of the batch
    table, n_pages = make_table(np.maximum(start, 0) + 1, page, seed=5)
    cache = J.paged_cache(n_pages, page, H, D, fmt)
    before = snapshot(cache)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(B, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    J.cache_append(cache, k.cuda(), v.cuda(), cu(table), cu(start))
    assert J.device_status() == 0
    same_bits(snapshot(cache), expect_append(before, table, page, start, np.arange(B + 1), k, v, fmt))


def test_append_quantises_every_range():
    """Blocks of all magnitudes (zero, subnormal, the largest bf16), ties between codes, saturating values, NaN and
    infinities: codes and exponents bit for bit."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    D, page = 128, 64
    rows = [torch.randn(D, generator=torch.Generator().manual_seed(i)) * 2.0**e for i, e in
            enumerate(list(range(-133, 127, 4)) + [127])]
    ties = torch.tensor([1.0 + (2 * i + 1) / 16 for i in range(8)] + [0.75 * 2.0**-9, 1.5 * 2.0**-9, 2.5 * 2.0**-9, 0.5 * 2.0**-9])
    special = torch.zeros(D)
    special[:12] = ties
    special[12] = 448.0
    special[32:44] = -ties
    special[44] = 511.0  # between 448 * 2^E and 512 * 2^E: saturates
    rows.append(special)
    bad = torch.randn(D, generator=torch.Generator().manual_seed(99))
    bad[3], bad[40], bad[100] = float("nan"), float("inf"), float("-inf")
    rows += [bad, torch.zeros(D)]
    x = torch.stack(rows).to(torch.bfloat16)[:, None, :].contiguous()
    n = x.shape[0]
    table, n_pages = make_table([n], page, 7)
    cache = J.paged_cache(n_pages, page, 1, D, "mxfp8")
    before = snapshot(cache)
    off = np.array([0, n])
    J.cache_append(cache, x.cuda(), (-x).cuda(), cu(table), cu(np.array([0])), off=cu(off))
    assert J.device_status() == 0
    same_bits(snapshot(cache), expect_append(before, table, page, np.array([0]), off, x, -x, "mxfp8"))
    # and read back: what the codes stand for, rounded to bf16 once
    k, v = J.cache_read(cache, cu(table), cu(off))
    codes, e = R.quantise(np64(x))
    want = torch.from_numpy(R.dequantise(codes, e)).to(torch.bfloat16)
    for got, w in ((k, want), (v, -want)):
        got = got.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(w, nan=0.0))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("D,page,H", [(128, 16, 3), (64, 8, 1), (64, 128, 2)])
def test_read_returns_cached_rows(D, page, H, fmt):
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens = [1, 40, 0, 129, 7]
    start = np.array([0, 13, 0, 100, -1])
    cache, table, pages = fill_cache(J, lens, page, H, D, fmt, seed=11)
    want = np.maximum(np.array(lens) - np.maximum(start, 0), 0)
    off = prefix(want)
    total = int(off[-1]) + 2
    k0 = torch.full((total, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    v0 = k0.clone()
    k, v = J.cache_read(cache, cu(table), cu(off), start=cu(start), k=k0, v=v0)
    assert k is k0 and v is v0 and J.device_status() == 0
    for got, pg in ((k, pages[0]), (v, pages[1])):
        got = np64(got)
        for b in range(len(lens)):
            rows = got[off[b]:off[b + 1]]
            if start[b] < 0:
                assert np.all(rows == 7.0)
            else:
                assert np.array_equal(rows, R.gather(pg, table, b, lens[b])[start[b]:])
        assert np.all(got[off[-1]:] == 7.0)  # rows behind the last sequence
    whole = prefix(lens)
    k2, _ = J.cache_read(cache, cu(table), cu(whole))  # start 0, total read from off
    assert np.array_equal(np64(k2), np.concatenate([R.gather(pages[0], table, b, n) for b, n in enumerate(lens)]))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_append_and_read_report_bad_places(fmt):
    """Bad pages, positions past the table, offsets that decrease, rotary positions past the tables: a status, no
    access outside the buffers, good rows done."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, D, page = 2, 64, 16
    x = torch.randn(6, H, D, device="cuda").to(torch.bfloat16)
    off = cu(np.array([0, 3, 6]))
    table = cu(np.array([[0, 1], [2, 3]], np.int32))
    cache = J.paged_cache(4, page, H, D, fmt)

    def run(code, table=table, start=(0, 0), off=off, rope=None):
        before = snapshot(cache)
        J.cache_append(cache, x, x, table, cu(np.array(start)), off=off, rope=rope)
        assert J.device_status() == code
        return before

    for bad in (4, -1, 2**31 - 1):
        b = run(PAGES, table=cu(np.array([[bad, 1], [2, 3]], np.int32)))
        assert torch.equal(cache.k[0], b[0][0]) and torch.equal(cache.k[1], b[0][1])
    b = run(LENGTH, start=(30, 0))  # rows 30, 31 fit, row 32 does not
    for s in (33, 2**31, 2**62):
        run(LENGTH, start=(s, 0))
    run(OFFSETS, off=cu(np.array([0, 5, 3])))
    run(OFFSETS, off=cu(np.array([2, 3, 6])))
    cos = torch.ones(2, D // 2, device="cuda")
    run(ROPE, rope=(cos, torch.zeros_like(cos)))
    k, v = J.cache_read(cache, cu(np.array([[9, 1], [2, 3]], np.int32)), off)
    assert J.device_status() == PAGES and bool((k[:3] == 0).all()) and bool((v[:3] == 0).all())
    J.cache_read(cache, table, off, start=cu(np.array([30, 0])))
    assert J.device_status() == LENGTH
    J.cache_read(cache, table, cu(np.array([0, 5, 3])), total=6)
    assert J.device_status() == OFFSETS
    run(0)
    k, _ = J.cache_read(cache, table, off)
    assert J.device_status() == 0 and (fmt == "mxfp8" or torch.equal(k, x))


# ------------------------------------------------------------------ decode
def weight_parts(fmt, spread=4):
    """MXFP8: weights are held in fp16 at 2^7 times their share of the row's largest and multiplied by their V block's
    2^-spread: half a step is 2^-11, or 2^-25 absolute below fp16's normal range, 2^(-25 - 7 + spread) of the largest.
    (Normal values: block maxima of 32 lie within 2^4.)"""
    return {} if fmt == "bf16" else dict(part=2.0**-11, floor=2.0 ** (spread - 32))


def check_decode(J, lens, lq, Hq, H, D, page, fmt, seed=21, act="softmax", causal=False, window=0, block=0, norm=False,
                 scale=None, extra_rows=0, max_kv=None, one_row=False):
    clear(J)
    std = 1.0 if act == "softmax" else 0.5
    cache, table, pages = fill_cache(J, lens, page, H, D, fmt, seed, extra_cols=1, std=std)
    q_off = prefix(lq)
    total = int(q_off[-1]) + extra_rows
    q = (torch.randn(total, Hq, D, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)
    out = torch.full((total, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse0 = torch.full((total, Hq), 5.0, device="cuda")
    kw = dict(act=act, causal=causal, window=window, block=block)
    o, lse = J.decode(q.cuda(), cache, cu(table), cu(np.asarray(lens, np.int64)), q_off=None if one_row else cu(q_off),
                      norm_by_lkv=norm, scale=scale, out=out, lse=lse0, max_kv=max_kv, **kw)
    assert J.device_status() == 0
    ro, rl, to, tl = R.decode(np64(q), pages[0], pages[1], table, lens, q_off, norm=norm, scale=scale,
                              **weight_parts(fmt), **kw)
    n = int(q_off[-1])
    go = np64(o)
    assert np.all(np.isfinite(go))
    worst = np.abs(go[:n] - ro[:n]) - to[:n]
    assert worst.max(initial=-1) <= 0, f"o off by {worst.max()} more than its bound"
    assert np.all(go[n:] == 5.0)
    if act == "softmax":
        gl = np64(lse)
        empty = np.isinf(rl[:n])
        assert np.array_equal(np.isinf(gl[:n]), empty)
        d = np.abs(gl[:n][~empty] - rl[:n][~empty]) - tl[:n][~empty]
        assert d.max(initial=-1) <= 0, f"lse off by {d.max()} more than its bound"
        assert np.all(gl[n:] == 5.0)
    else:
        assert lse is None
    return o, lse


LENS = [1, 17, 0, 64, 130, 259, 3, 16]


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("D,page", [(128, 16), (128, 64), (64, 8), (64, 128)])
@pytest.mark.parametrize("Hq,H", [(2, 2), (6, 2), (8, 1), (20, 1), (3, 3)])
def test_decode_single_rows(Hq, H, D, page, fmt):
    import jagged_attention_recsys_gdpa_gb300 as J

    check_decode(J, LENS, [1] * len(LENS), Hq, H, D, page, fmt, one_row=True)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("act,norm", [("softmax", False), ("silu", True), ("silu", False), ("gelu", True),
                                      ("gelu", False), ("gelu_poly", True)])
@pytest.mark.parametrize("mask", [{}, dict(causal=True), dict(causal=True, window=20), dict(block=16),
                                  dict(block=48, causal=True)], ids=["none", "causal", "window", "block", "cblock"])
def test_decode_rows_masks_activations(act, norm, mask, fmt):
    """Several query rows per sequence (none, and more than there are keys), all masks: rows that see nothing give
    zeros and -inf, rows behind the last sequence stay as they were."""
    import jagged_attention_recsys_gdpa_gb300 as J

    lq = [1, 5, 2, 3, 0, 7, 6, 17]
    poly = dict(scale=0.04) if act == "gelu_poly" else {}
    check_decode(J, LENS, lq, 4, 2, 128, 32, fmt, act=act, norm=norm, extra_rows=2, **mask, **poly)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H,lq", [(1, 1, 33), (8, 2, 13), (4, 4, 70), (16, 1, 5)])
def test_decode_many_rows(Hq, H, lq, D, fmt):
    """More rows per key/value head than one tile of the kernel holds."""
    import jagged_attention_recsys_gdpa_gb300 as J

    check_decode(J, [90, 200, 5], [lq, 1, lq], Hq, H, D, 16, fmt, causal=True, seed=31)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("lens", [[4000], [2500, 1, 700, 0], [300] * 40])
def test_decode_long_lengths(lens, fmt):
    """Lengths that are split over many workers and joined."""
    import jagged_attention_recsys_gdpa_gb300 as J

    check_decode(J, lens, [1] * len(lens), 2, 1, 128, 64, fmt, seed=41, one_row=True)
    check_decode(J, lens, [2] * len(lens), 2, 2, 64, 64, fmt, seed=42, causal=True, window=333)
    check_decode(J, lens, [3] * len(lens), 3, 1, 128, 16, fmt, seed=43, act="silu", norm=True)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_decode_many_sequences(fmt):
    """More sequences than a CTA has threads (the plan then counts stretches of them), most of them short or empty."""
    import jagged_attention_recsys_gdpa_gb300 as J

    rng = np.random.default_rng(44)
    lens = (rng.integers(0, 40, 300) * (rng.random(300) < 0.8)).tolist()
    check_decode(J, lens, rng.integers(0, 3, 300).tolist(), 2, 1, 64, 16, fmt, seed=45, causal=True)
    lens = (rng.integers(0, 3, 5000) * (rng.random(5000) < 0.3)).tolist()
    check_decode(J, lens, [1] * 5000, 1, 1, 64, 8, fmt, seed=46, one_row=True)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_many_tiles(D, fmt):
    """Several tiles of rows per key/value head: of many sequences with few rows each, and of a long history whose
    tiles are each split over workers and joined."""
    import jagged_attention_recsys_gdpa_gb300 as J

    rng = np.random.default_rng(71)
    lens = rng.integers(0, 30, 200).tolist()
    check_decode(J, lens, rng.integers(0, 9, 200).tolist(), 6, 2, D, 16, fmt, seed=72, causal=True, extra_rows=1)
    check_decode(J, [2500, 0, 90], [25, 3, 1], 6, 3, D, 64, fmt, seed=73, causal=True, window=2000)
    check_decode(J, [1300, 700], [50, 3], 2, 2, D, 8, fmt, seed=74, act="silu", norm=True)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_decode_empty_calls(fmt):
    """No query rows at all; a bound of no cached rows; sequences that share their pages."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    cache, table, pages = fill_cache(J, [40, 70], 16, 2, 64, fmt, seed=47)
    none = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = J.decode(none, cache, cu(table), cu(np.array([40, 70])), q_off=cu(np.zeros(3, np.int64)))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    o, lse = J.decode(q, cache, cu(table), cu(np.zeros(2, np.int64)), max_kv=0)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    both = np.stack([table[1], table[1]])
    same = q[:1].expand(2, -1, -1).contiguous()
    o, lse = J.decode(same, cache, cu(both), cu(np.array([70, 70])))
    # The two sequences lie at different places of the split over workers, so their sums of the same terms are joined
    # from different pieces: (l0 + l1) + l2 in one, l0 + (l1 + l2) in the other, each with factors 2^(m_i - m) of its
    # own. A last bit of l, 2^-23 of it, is 2^-23 absolute in the lse and up to a step of o's rounding, so the two
    # need not be the same bit for bit; either has to lie within the bounds of the 64-bit values.
    ro, rl, to, tl = R.decode(np64(same), pages[0], pages[1], both, [70, 70], np.arange(3), **weight_parts(fmt))
    assert np.all(np.abs(np64(o) - ro) <= to) and np.all(np.abs(np64(lse) - rl) <= tl)
    x = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    J.cache_append(cache, x, x, cu(table), cu(np.zeros(2, np.int64)), off=cu(np.zeros(3, np.int64)))
    k, v = J.cache_read(cache, cu(table), cu(np.zeros(3, np.int64)))
    assert k.shape == v.shape == (0, 2, 64)
    assert J.device_status() == 0


def test_expired_wait_reports_timeout_and_context_survives():
    """Every worker's first copy skipped: the bounded waits run out, the call returns and the next one is right."""
    import jagged_attention_recsys_gdpa_gb300 as J
    from jagged_attention_recsys_gdpa_gb300 import _binding as B

    clear(J)
    for Hq, fmt in ((2, "bf16"), (24, "mxfp8"), (64, "bf16")):  # one warp a worker, three tiles a head, two warps a worker
        cache, table, _ = fill_cache(J, [400, 70, 3], 16, 1, 128, fmt, seed=48)
        q = torch.randn(3, Hq, 128, device="cuda").to(torch.bfloat16)
        args = (q, cache, cu(table), cu(np.array([400, 70, 3])))
        o, lse = J.decode(*args)
        torch.cuda.synchronize()
        try:
            B.debug_set(1, 20_000_000)
            J.decode(*args)
            assert J.device_status() == 6
        finally:
            B.debug_set(0, 0)
        o2, lse2 = J.decode(*args)
        assert J.device_status() == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_rows_at_16_byte_addresses(fmt):
    """Tensors whose first row lies 16 bytes behind a 32-byte boundary; 2 bytes behind one is refused."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, D, page, n = 2, 64, 16, 37
    flat = torch.randn(2 * n * H * D + 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    at = lambda t, o: t[o:o + n * H * D].view(n, H, D)  # noqa: E731
    k, v = at(flat, 8), at(flat, 8 + n * H * D + 16)
    assert k.data_ptr() % 32 == 16 and v.data_ptr() % 32 == 16
    table, n_pages = make_table([n], page, 6)
    off, start = cu(np.array([0, n])), cu(np.array([0]))
    caches = [J.paged_cache(n_pages, page, H, D, fmt) for _ in range(2)]
    J.cache_append(caches[0], k, v, cu(table), start, off=off)
    J.cache_append(caches[1], k.clone(), v.clone(), cu(table), start, off=off)
    same_bits(snapshot(caches[0]), [None if t is None else t.cpu() for t in snapshot(caches[1])])
    out = torch.zeros_like(flat)
    J.cache_read(caches[0], cu(table), off, k=at(out, 8), v=at(out, 8 + n * H * D + 16))
    want = J.cache_read(caches[0], cu(table), off)
    assert torch.equal(at(out, 8), want[0]) and torch.equal(at(out, 8 + n * H * D + 16), want[1])
    assert J.device_status() == 0
    with pytest.raises(J.JattnError):
        J.cache_append(caches[0], at(flat, 1), v, cu(table), start, off=off)
    with pytest.raises(J.JattnError):
        J.cache_read(caches[0], cu(table), off, k=at(out, 1), v=at(out, 8 + n * H * D + 16))
    with pytest.raises(J.JattnError):
        J.decode(at(flat, 1), caches[0], cu(np.repeat(table, n, 0)), torch.ones(n, dtype=torch.int64, device="cuda"))


def test_first_call_inside_a_capture_is_refused(monkeypatch):
    import jagged_attention_recsys_gdpa_gb300 as J
    from jagged_attention_recsys_gdpa_gb300 import paged

    cache = J.paged_cache(2, 16, 1, 64)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int64, device="cuda")
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    J.decode(q, cache, table, lens)
    monkeypatch.setattr(paged, "_status_blocks", {})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.add_(0)
        with pytest.raises(RuntimeError, match="before the capture"):
            J.decode(q, cache, table, lens)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_decode_large_scores(fmt):
    """Peaked softmax: score differences of hundreds, a maximum that moves along the length."""
    import jagged_attention_recsys_gdpa_gb300 as J

    check_decode(J, [1000, 37], [2, 1], 4, 2, 128, 32, fmt, scale=3.0, causal=True, seed=51)


@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("case", ["v_blocks", "v_grows", "v_huge", "v_tiny", "v_zero", "q_rows", "k_huge"])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_mxfp8_dynamic_range(case, act, D):
    """MXFP8 caches whose blocks lie many powers of two apart (within a row, along the sequence, near both ends of the
    exponents), and query rows far from 1."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, Hq, page, lens = 2, 4, 32, [200, 33, 1, 70]
    cache, table, pages = fill_cache(J, lens, page, H, D, "mxfp8", seed=101)
    rng = np.random.default_rng(102)
    ke, ve = cache.k_scales, cache.v_scales
    shift = {"v_blocks": lambda: torch.randint(-40, 3, ve.shape, device="cuda"),
             "v_grows": lambda: torch.arange(ve.shape[0] * page, device="cuda").view(-1, 1, page, 1) // 4,
             "v_huge": lambda: torch.randint(0, 90, ve.shape, device="cuda"),
             "v_tiny": lambda: torch.randint(-119, -60, ve.shape, device="cuda"),
             "v_zero": lambda: -1000 * (torch.rand(ve.shape, device="cuda") < 0.3)}.get(case)
    live = (ve != 255).clone()
    if shift is not None:
        torch.manual_seed(5)
        moved = (ve.int() + shift()).clamp(0, 246).to(torch.uint8)
        ve.copy_(torch.where(live, moved, ve))
        if case == "v_zero":
            dead = (ve == 0).repeat_interleave(32, -1)
            cache.v[dead] = 0
    q = torch.randn(4, Hq, D, generator=torch.Generator().manual_seed(3))
    kw = dict(act=act)
    if case == "k_huge":
        ke.copy_(torch.where(live, ke + 60, ke))
        q = q * 2.0**-60
    if case == "q_rows":
        q = q * torch.tensor([2.0**-125, 1e-3, 1.0, 2.0**10])[:, None, None]
        kw["scale"] = 2.0**-8
    q = q.to(torch.bfloat16)
    # the pages' values again, from the exponents as they are now (NaN places are never live)
    kp, vp = (np.nan_to_num(R.dequantise(c.cpu().numpy(), e.cpu().numpy())) for c, e in ((cache.k, ke), (cache.v, ve)))
    o, lse = J.decode(q.cuda(), cache, cu(table), cu(np.array(lens)), **kw)
    assert J.device_status() == 0
    # V blocks may lie 2^14 below the unit's largest (below that, bf16 products hold the weights in two parts)
    ro, rl, to, tl = R.decode(np64(q), kp, vp, table, lens, np.arange(5), **weight_parts("mxfp8", 14), **kw)
    # bf16 subnormals: half a step of 2^-133; scores and values this far down underflow in fp32 terms of 2^-126 each
    floor = 2.0**-134 + 200 * 2.0**-126
    top = float(torch.finfo(torch.bfloat16).max)
    over = np.abs(ro) > top  # beyond bf16 (sums of unscaled weights): infinity, of the same sign
    assert np.all((np64(o)[over] == np.sign(ro[over]) * np.inf) | (np.abs(np64(o)[over] - ro[over]) <= to[over]))
    assert np.all(np.abs(np64(o) - ro)[~over] <= (to + floor)[~over])
    if act == "softmax":
        assert np.all(np.abs(np64(lse) - rl) <= tl)


def test_decode_mxfp8_largest_exponent():
    """V blocks of exponent 254 (the largest number E8M0 has) with codes small enough for finite sums: values up to
    7 * 2^-9 * 2^127, averaged by softmax weights."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, D, page, lens = 2, 128, 32, [200, 33, 1, 70]
    cache, table, _ = fill_cache(J, lens, page, H, D, "mxfp8", seed=111)
    g = torch.Generator().manual_seed(112)
    sign = torch.randint(0, 2, cache.v.shape, generator=g) * 128
    cache.v.copy_((torch.randint(0, 8, cache.v.shape, generator=g) + sign).to(torch.uint8))
    cache.v_scales.copy_((254 - torch.randint(0, 4, cache.v_scales.shape, generator=g)).to(torch.uint8))
    q = torch.randn(4, 2 * H, D, generator=g).to(torch.bfloat16)
    o, _ = J.decode(q.cuda(), cache, cu(table), cu(np.array(lens)))
    assert J.device_status() == 0
    kp, vp = (R.dequantise(c.cpu().numpy(), e.cpu().numpy())
              for c, e in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)))
    ro, _, to, _ = R.decode(np64(q), np.nan_to_num(kp), vp, table, lens, np.arange(5), **weight_parts("mxfp8", 4))
    assert np.all(np.abs(np64(o) - ro) <= to)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("H,D,total", [(1, 64, 1_300_007), (8, 128, 83_001)])
def test_large_calls_do_what_small_ones_do(H, D, total, fmt):
    """Calls large enough for several rows and batches a thread against calls of one unit a thread (which the tests above
    hold to the definitions), bit for bit."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    B, page = 37, 64
    g = torch.Generator().manual_seed(61)
    lens = torch.rand(B, generator=g) + 0.05
    lens = (lens / lens.sum() * total).long()
    lens[5] = 0
    lens[-1] += total - lens.sum()
    off = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    need = (lens + page - 1) // page
    table = torch.zeros(B, int(need.max()), dtype=torch.int32)
    pages = torch.randperm(int(need.sum()), generator=g).int()
    at = 0
    for b in range(B):
        table[b, :need[b]] = pages[at:at + int(need[b])]
        at += int(need[b])
    k, v = (torch.randn(total, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    rope = tuple(torch.randn(int(lens.max()), D // 2, device="cuda") for _ in range(2))
    many, one = (J.paged_cache(len(pages), page, H, D, fmt) for _ in range(2))
    zero = torch.zeros(B, dtype=torch.int64, device="cuda")
    J.cache_append(one, k, v, table.cuda(), zero, off=off.cuda(), rope=rope)
    ko, vo = J.cache_read(one, table.cuda(), off.cuda())
    piece = 300_000 // (H * D // 8)  # rows: fewer than 311,296 units of 8 (or 16) values
    for b in range(B):
        for first in range(0, int(lens[b]), piece):
            n = min(piece, int(lens[b]) - first)
            rows = slice(int(off[b]) + first, int(off[b]) + first + n)
            start, o = torch.tensor([first], device="cuda"), torch.tensor([0, n], device="cuda")
            J.cache_append(many, k[rows], v[rows], table[b:b + 1].cuda(), start, off=o, rope=rope)
            kr, vr = J.cache_read(many, table[b:b + 1].cuda(), o, start=start)
            assert torch.equal(kr, ko[rows]) and torch.equal(vr, vo[rows])
    assert J.device_status() == 0
    for x, y in ((one.k, many.k), (one.v, many.v), (one.k_scales, many.k_scales), (one.v_scales, many.v_scales)):
        assert x is None and y is None or torch.equal(x, y)


def test_append_refuses_rows_that_need_a_gradient():
    import jagged_attention_recsys_gdpa_gb300 as J

    cache = J.paged_cache(2, 16, 2, 64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int64, device="cuda")
    x = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
    y = x.clone().requires_grad_(True)
    for k, v in ((y, x), (x, y)):
        with pytest.raises(ValueError, match="no backward pass"):
            J.cache_append(cache, k, v, table, start)
    with torch.no_grad():
        J.cache_append(cache, y, y, table, start)
    assert torch.equal(cache.k[0, :, 0], x[0])


def test_decode_masked_values_never_reach_a_row():
    """Infinities and NaN in K and V at positions that only later rows may see."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, D, page, n, lq = 2, 128, 16, 50, 4
    q = torch.randn(lq, H, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q_off = np.array([0, lq])
    for mask in (dict(causal=True), dict(causal=True, window=5), dict(block=49)):
        cache, table, pages = fill_cache(J, [n], page, H, D, "bf16", seed=61)
        want, _, tol, _ = R.decode(np64(q), pages[0], pages[1], table, [n], q_off, **mask)
        args = (cu(table), cu(np.array([n])))
        clean, lse_clean = J.decode(q, cache, *args, q_off=cu(q_off), **mask)
        last = n - 1  # seen by the last row alone (block 49: the last row's block)
        at = (int(table[0, last // page]), slice(None), last % page, slice(5, 90))
        for kind, value in ((k, x) for k in "kv" for x in (float("nan"), float("inf"), float("-inf"))):
            buf = cache.k if kind == "k" else cache.v
            saved = buf[at].clone()
            buf[at] = value
            o, lse = J.decode(q, cache, *args, q_off=cu(q_off), **mask)
            buf[at] = saved
            assert J.device_status() == 0
            assert torch.equal(lse[:-1], lse_clean[:-1])
            if kind == "k":
                assert torch.equal(o[:-1], clean[:-1]), (value, mask)
                continue
            # the columns that hold the value are summed in another order for the rows that do not see it (within the
            # bound all the same); the row that sees it has it there, and every other column is as it was
            assert np.all(np.abs(np64(o)[:-1] - want[:-1]) <= tol[:-1]), (value, mask)
            assert not bool(torch.isfinite(o[-1, :, 5:90]).any())
            assert torch.equal(lse, lse_clean)
            assert torch.equal(o[..., :5], clean[..., :5]) and torch.equal(o[..., 90:], clean[..., 90:])


def test_decode_reports_bad_inputs():
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens = [40, 70]
    cache, table, _ = fill_cache(J, lens, 16, 2, 64, "bf16", seed=71)
    q = torch.randn(2, 2, 64, device="cuda").to(torch.bfloat16)
    good, _ = J.decode(q, cache, cu(table), cu(np.array(lens)))
    assert J.device_status() == 0
    for bad in (-1, 2**31 - 1, cache.n_pages):
        t = table.copy()
        t[1, 2] = bad
        o, _ = J.decode(q, cache, cu(t), cu(np.array(lens)))
        assert J.device_status() == PAGES
        assert torch.equal(o[0], good[0])
    for n in (-1, 16 * table.shape[1] + 1, 2**40, -2**62):
        o, lse = J.decode(q, cache, cu(table), cu(np.array([40, n])))
        assert J.device_status() == LENGTH
        assert torch.equal(o[0], good[0]) and bool((o[1] == 0).all()) and bool(torch.isinf(lse[1]).all())
    o, _ = J.decode(q, cache, cu(table), cu(np.array(lens)), max_kv=50)
    assert J.device_status() == LENGTH
    for off in ([0, 2, 1], [0, 1, 3], [1, 1, 2], [0, 2**40, 2], [-5, 1, 2]):
        J.decode(q, cache, cu(table), cu(np.array(lens)), q_off=cu(np.array(off)))
        assert J.device_status() == OFFSETS, off
    o, _ = J.decode(q, cache, cu(table), cu(np.array(lens)))
    assert J.device_status() == 0 and torch.equal(o, good)


def test_decode_is_the_same_from_call_to_call_and_stream_to_stream():
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens = [3000, 5, 900, 0, 1200]
    cache, table, _ = fill_cache(J, lens, 32, 2, 128, "mxfp8", seed=81)
    q = torch.randn(5, 8, 128, device="cuda").to(torch.bfloat16)
    args = (cache, cu(table), cu(np.array(lens)))
    o, lse = J.decode(q, *args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(30):  # calls that run at the same time
        with torch.cuda.stream(streams[i % 3]):
            got.append(J.decode(q, *args))
    torch.cuda.synchronize()
    assert J.device_status() == 0
    for a, b in got:
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_captured_graphs_replay_with_new_lengths():
    """Two captured decode steps (append, then attention) replayed at the same time on two streams, with lengths, rows
    and tables changed in place between replays."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, D, page, B, cap = 2, 128, 16, 4, 256
    rng = np.random.default_rng(91)
    sides = []
    for i in range(2):
        cache = J.paged_cache(B * cap // page, page, H, D, "mxfp8" if i else "bf16")
        table = cu(rng.permutation(B * cap // page).reshape(B, -1).astype(np.int32))
        start = torch.zeros(B, dtype=torch.int64, device="cuda")
        x = [torch.zeros(B, h, D, dtype=torch.bfloat16, device="cuda") for h in (2 * H, H, H)]
        out, lse = torch.empty_like(x[0]), torch.empty(B, 2 * H, device="cuda")

        def step(cache=cache, table=table, start=start, x=x, out=out, lse=lse):
            J.cache_append(cache, x[1], x[2], table, start)
            J.decode(x[0], cache, table, start + 1, out=out, lse=lse)

        step()  # warm-up outside the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        sides.append((cache, table, start, x, out, lse, graph, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for t in range(40):
        for i, (cache, table, start, x, out, lse, graph, st) in enumerate(sides):
            with torch.cuda.stream(st):
                for y in x:
                    y.copy_(torch.randn(y.shape, generator=torch.Generator().manual_seed(1000 * i + t)).to(torch.bfloat16))
                start.fill_(t)
                graph.replay()
    torch.cuda.synchronize()
    assert J.device_status() == 0
    for i, (cache, table, start, x, out, lse, graph, st) in enumerate(sides):
        o, l2 = J.decode(x[0], cache, table, start + 1)
        assert torch.equal(o, out) and torch.equal(l2, lse)
        k, _ = J.cache_read(cache, table, cu(prefix([40] * B)))
        # the generator gives each of x's tensors the same stream of numbers: rows of the last step
        want = torch.randn((B, H, D), generator=torch.Generator().manual_seed(1000 * i + 39)).to(torch.bfloat16)
        if i == 0:
            assert torch.equal(k.view(B, 40, H, D)[:, 39].cpu(), want)


def test_pages_beyond_32_bit_offsets():
    """A cache of more than 2^32 elements: pages at its far end."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, D, page = 8, 128, 64
    n_pages = (2**32 // (H * page * D)) + 40
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * n_pages * H * page * D * 2:
        pytest.skip("not enough free memory")
    for fmt in ("bf16", "mxfp8"):
        small, table, pages = fill_cache(J, [100, 65], page, H, D, fmt, seed=95)
        big = J.paged_cache(n_pages, page, H, D, fmt)
        shift = n_pages - small.n_pages
        for dst, src in ((big.k, small.k), (big.v, small.v), (big.k_scales, small.k_scales), (big.v_scales, small.v_scales)):
            if src is not None:
                dst[shift:] = src
        far = np.where(table < 0, table, table + shift).astype(np.int32)
        q = torch.randn(2, H, D, device="cuda").to(torch.bfloat16)
        o, lse = J.decode(q, small, cu(table), cu(np.array([100, 65])))
        o2, lse2 = J.decode(q, big, cu(far), cu(np.array([100, 65])))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        off = cu(prefix([100, 65]))
        k, v = J.cache_read(big, cu(far), off)
        k0, v0 = J.cache_read(small, cu(table), off)
        assert torch.equal(k, k0) and torch.equal(v, v0)
        J.cache_append(big, k, v, cu(far), cu(np.zeros(2, np.int64)), off=off)
        assert J.device_status() == 0
        assert torch.equal(big.k[shift:][small.k == small.k], small.k[small.k == small.k]) or fmt == "mxfp8"
        del big


# ------------------------------------------------------------------ together
def test_serving_a_jagged_model_step_by_step():
    """Prompts through the jagged forward and the cache, then new rows one at a time: every step's output agrees with
    the jagged forward over the whole sequences, and a chunk read back from the cache continues a prompt."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, D, page, steps = 4, 128, 16, 5
    prompt = np.array([40, 1, 130, 15])
    whole = prompt + steps
    B = len(prompt)
    g = torch.Generator(device="cuda").manual_seed(7)
    full = [torch.randn(int(whole.sum()), H, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    cos, sin, _ = rope_tables(256, D)
    rope = (cu(cos.astype(np.float32)), cu(sin.astype(np.float32)))
    w_off = prefix(whole)
    wo = cu(w_off)
    q_rot = J.rope(full[0], wo, wo, rope)
    k_rot = J.rope(full[1], wo, wo, rope, keys=True)
    want, want_lse = J.forward(q_rot, k_rot, full[2], wo, wo, causal=True)
    table, n_pages = make_table(whole, page, 8)
    table = cu(table)
    cache = J.paged_cache(n_pages, page, H, D, "bf16")
    rows = torch.cat([torch.arange(w_off[b], w_off[b] + prompt[b]) for b in range(B)]).cuda()
    J.cache_append(cache, full[1][rows], full[2][rows], table, torch.zeros(B, dtype=torch.int64, device="cuda"),
                   off=cu(prefix(prompt)), rope=rope)
    for t in range(steps):
        lens = cu(prompt + t)
        new = cu(w_off[:-1] + prompt + t)
        J.cache_append(cache, full[1][new], full[2][new], table, lens, rope=rope)
        o, lse = J.decode(q_rot[new], cache, table, lens + 1)
        assert torch.allclose(o.float(), want[new].float(), atol=1e-2, rtol=1e-2)
        assert torch.allclose(lse, want_lse[new], atol=1e-3)
    # the last rows as one chunk: keys and values read back, queries at the sequences' ends
    k, v = J.cache_read(cache, table, wo)
    assert torch.equal(v, full[2])
    tail = torch.cat([torch.arange(w_off[b] + prompt[b], w_off[b + 1]) for b in range(B)]).cuda()
    t_off = cu(prefix([steps] * B))
    o, _ = J.forward(q_rot[tail].contiguous(), k, v, t_off, wo, causal=True)
    assert torch.allclose(o.float(), want[tail].float(), atol=1e-2, rtol=1e-2)
    od, _ = J.decode(q_rot[tail].contiguous(), cache, table, cu(whole), q_off=t_off, causal=True)
    assert torch.allclose(od.float(), o.float(), atol=1e-2, rtol=1e-2)
    assert J.device_status() == 0


def test_python_refusals():
    import jagged_attention_recsys_gdpa_gb300 as J

    cache = J.paged_cache(4, 16, 2, 64)
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int64, device="cuda")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    J.decode(q, cache, table, lens)
    bad = [dict(q=q.float()), dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q.transpose(0, 1)), dict(q=q.cpu()),
           dict(table=table.long()), dict(table=table[:, :0]), dict(table=torch.zeros(2, 3, dtype=torch.int32, device="cuda")[:, :2]), dict(lens=lens.int()),
           dict(lens=lens[:1]), dict(lens=lens.cpu()), dict(q_off=lens), dict(max_kv=33), dict(max_kv=-1),
           dict(out=x), dict(lse=lens), dict(window=2, block=2), dict(q=q.clone().requires_grad_(True))]
    for kw in bad:
        kw = dict(dict(q=q, table=table, lens=lens), **kw)
        with pytest.raises(ValueError):
            J.decode(kw.pop("q"), cache, kw.pop("table"), kw.pop("lens"), **kw)
    with torch.no_grad():
        J.decode(q.clone().requires_grad_(True), cache, table, lens)
    for kw in (dict(k=x[:1]), dict(k=x.float()), dict(start=lens.int()), dict(table=table.long()), dict(off=lens)):
        kw = dict(dict(k=x, table=table, start=lens, off=None), **kw)
        with pytest.raises(ValueError):
            J.cache_append(cache, kw["k"], x, kw["table"], kw["start"], off=kw["off"])
    with pytest.raises(ValueError):
        J.cache_read(cache, table, lens)
    for kw in (dict(page_size=24), dict(page_size=4), dict(D=96), dict(format="fp8"), dict(page_size=8192)):
        with pytest.raises(ValueError):
            J.paged_cache(**dict(dict(n_pages=2, page_size=16, H=2, D=64), **kw))
    with pytest.raises(ValueError):
        J.PagedCache(cache.k, cache.v, torch.zeros(1, dtype=torch.uint8, device="cuda"), None)
