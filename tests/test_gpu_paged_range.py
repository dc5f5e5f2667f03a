"""Decode from MXFP8 caches whose V exponents lie far apart, between the units
that one worker takes one after another and within one unit, and NaN blocks and
codes, against the plain 64-bit reference in paged_ref."""
import numpy as np
import pytest
import torch

from tests import paged_ref as R
from tests.test_gpu_paged import clear, cu, fill_cache, np64, prefix, weight_parts

pytestmark = pytest.mark.gpu


def pages_of(cache):
    """The float64 pages as they are now (NaN places become zeros: they lie in no sequence)."""
    return [np.nan_to_num(R.dequantise(c.cpu().numpy(), e.cpu().numpy()))
            for c, e in ((cache.k, cache.k_scales), (cache.v, cache.v_scales))]


def shift_values(cache, by):
    """V exponents moved by `by` (broadcast); the NaN places stay."""
    e = cache.v_scales
    e.copy_(torch.where(e == 255, e, (e.int() + by).clamp(0, 254).to(torch.uint8)))


def rows_of(table, lens, page):
    """(sequence, position, page, place in it) of every cached row."""
    for b, n in enumerate(lens):
        for p in range(int(n)):
            yield b, p, int(table[b, p // page]), p % page


def check_repeated(J, cache, table, lens, lq, Hq, rep, spread=4, seed=7, act="softmax", **mask):
    """The sequences `rep` times over in one call, all copies reading the same pages: every copy within the bounds of
    the 64-bit values."""
    D = cache.D
    q_off = prefix(lq)
    n = int(q_off[-1])
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    kp, vp = pages_of(cache)
    ro, rl, to, tl = R.decode(np64(q), kp, vp, table, lens, q_off, act=act, **weight_parts("mxfp8", spread), **mask)
    many = torch.from_numpy(np.concatenate([q_off[:-1] + i * n for i in range(rep)] + [[rep * n]])).cuda()
    o, lse = J.decode(q.cuda().repeat(rep, 1, 1), cache, cu(np.tile(table, (rep, 1))),
                      cu(np.tile(np.asarray(lens, np.int64), rep)), q_off=many, act=act, **mask)
    assert J.device_status() == 0
    ro, to = cu(ro), cu(to)
    for i in range(0, rep, 32):
        got = o[i * n:(i + 32) * n].view(-1, n, Hq, D).double()
        worst = ((got - ro).abs() - to).amax(dim=(2, 3))
        assert not bool(torch.isnan(got).any()) and float(worst.max()) <= 0, \
            f"copies {i}..: o off by {float(worst.max())} more than its bound, first at {(worst > 0).nonzero()[:4].tolist()}"
    if act == "softmax":
        off = (lse.view(rep, n, Hq).double() - cu(rl)).abs() - cu(tl)
        assert float(off.max()) <= 0


@pytest.mark.parametrize("D,rep,act", [(64, 1024, "softmax"), (64, 1024, "silu"), (128, 768, "softmax")])
def test_units_with_zero_blocks_leave_the_ones_behind_them_alone(D, rep, act):
    """Thousands of histories shorter than one product block, 64 query rows a head, so that a worker takes hundreds of
    units; some V rows are zeros (exponent 0), and the heads' values lie 2^8 apart."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens, page, H = [20, 1, 31, 7, 20, 24, 13, 25], 32, 8
    cache, table, _ = fill_cache(J, lens, page, H, D, "mxfp8", seed=201)
    shift_values(cache, (8 * (torch.arange(H, device="cuda") % 3)).view(1, H, 1, 1))
    for b, p, pg, at in rows_of(table, lens, page):
        if b % 4 == 0 and p % 5 == 2:
            cache.v[pg, :, at], cache.v_scales[pg, :, at] = 0, 0
    check_repeated(J, cache, table, lens, [1] * len(lens), 64 * H, rep, act=act)


@pytest.mark.parametrize("mask", [{}, dict(causal=True, window=20), dict(causal=True, block=24)],
                         ids=["none", "window", "block"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("act", ["softmax", "gelu"])
def test_a_neighbours_large_values_stay_its_own(act, D, mask):
    """Every other history's values are 2^130 times larger: the ones between them, short or behind a window that begins
    inside a product block, alone and in a batch of several units a worker."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens, page, H = [25, 21, 12, 30] if not mask else [75, 130, 90, 61], 16, 2
    cache, table, _ = fill_cache(J, lens, page, H, D, "mxfp8", seed=211)
    for b, p, pg, at in rows_of(table, lens, page):
        e = cache.v_scales[pg, :, at]
        cache.v_scales[pg, :, at] = (e.int() + (70 if b % 2 == 0 else -60)).to(torch.uint8)
    lq = [1, 2, 1, 3]
    check_repeated(J, cache, table, lens, lq, 4 * H, 1000, act=act, **mask)
    for b in (1, 3):
        check_repeated(J, cache, table[b:b + 1], lens[b:b + 1], lq[b:b + 1], 4 * H, 1, act=act, **mask)


@pytest.mark.parametrize("top", [120, 240, 252, 253, 254])
def test_a_nan_block_is_nan_beside_the_largest_exponents(top):
    """A block of exponent 255 (with codes of zero, as append writes it) among blocks up to the largest exponent: its 32
    columns are NaN for the rows that see it, everything else is as it has to be."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens, page, H, D = [90, 40], 32, 2, 128
    cache, table, _ = fill_cache(J, lens, page, H, D, "mxfp8", seed=221)
    g = torch.Generator().manual_seed(222)
    sign = torch.randint(0, 2, cache.v.shape, generator=g) * 128  # codes up to 7 * 2^-9: finite sums
    cache.v.copy_((torch.randint(0, 8, cache.v.shape, generator=g) + sign).to(torch.uint8))
    cache.v_scales.copy_((top - torch.randint(0, 4, cache.v_scales.shape, generator=g)).to(torch.uint8))
    cache.v_scales[table[0, 1], 1, 5, 1] = top
    kp, vp = pages_of(cache)
    q = torch.randn(3, 2 * H, D, generator=g).to(torch.bfloat16)
    q_off = np.array([0, 2, 3])
    ro, rl, to, tl = R.decode(np64(q), kp, vp, table, lens, q_off, causal=True, **weight_parts("mxfp8", 4))
    bad = (int(table[0, 89 // page]), 1, 89 % page, 2)  # the last key: the second row of the sequence alone sees it
    cache.v_scales[bad] = 255
    cache.v[bad[0], 1, bad[2], 64:96] = 0
    o, lse = J.decode(q.cuda(), cache, cu(table), cu(np.array(lens)), q_off=cu(q_off), causal=True)
    assert J.device_status() == 0
    got = np64(o)
    assert np.all(np.isnan(got[1, 2:, 64:96]))
    keep = np.ones(got.shape, bool)
    keep[1, 2:, 64:96] = False
    assert np.all(np.abs(got - ro)[keep] <= to[keep])
    assert np.all(np.abs(np64(lse) - rl) <= tl)


MASKS = {"causal": dict(causal=True), "window": dict(causal=True, window=60), "block": dict(block=49)}


@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("mask", sorted(MASKS))
@pytest.mark.parametrize("D", [64, 128])
def test_large_values_that_other_rows_see(D, mask, act):
    """Finite values up to 2^150 times a row's own at positions that only other rows of its tile see, at the end (one more
    for each row), at the start of a window and in another block: every row within the bound of the keys that it sees."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens, page, H, lq = [150, 40], 32, 2, [4, 3]
    for places in ("ends", "early") if mask == "window" else ("ends",):
        cache, table, _ = fill_cache(J, lens, page, H, D, "mxfp8", seed=231)
        shift_values(cache, -30)
        kw = MASKS[mask]
        for b, n in enumerate(lens):
            if places == "early":
                where = [(max(n - lq[b] - 59, 0) + i, e) for i, e in enumerate((239, 200, 160)[:lq[b] - 1])]
            elif mask == "block":
                where = [(p, 239) for p in range((n - 1) // 49 * 49, n)] if (n - lq[b]) // 49 != (n - 1) // 49 else []
            else:
                where = [(n - 1 - i, e) for i, e in enumerate((239, 200, 160)[:lq[b] - 1])]
            for p, e in where:
                cache.v_scales[int(table[b, p // page]), :, p % page] = e
        check_repeated(J, cache, table, lens, lq, 2 * H, 3, spread=14, act=act, **kw)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("at", [3, 60, 99])
def test_large_values_whose_weight_vanishes(at, fmt):
    """A key whose softmax weight is 2^-450 or less and whose values are 2^120 times the others' or more: it adds nothing, and
    takes nothing away."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens, page, H, D = [100], 32, 2, 128
    cache, table, _ = fill_cache(J, lens, page, H, D, fmt, seed=241)
    pg, row = int(table[0, at // page]), at % page
    q = (torch.rand(1, H, D, generator=torch.Generator().manual_seed(4)) + 1.0).to(torch.bfloat16)
    if fmt == "mxfp8":  # keys of -448 / 2^4 against queries between 1 and 2: a score of -316 or less
        cache.k[pg, :, row], cache.k_scales[pg, :, row] = 0xfe, 123
        kp, vp = pages_of(cache)
    else:
        cache.k[pg, :, row] = -28.0
        kp, vp = (np.nan_to_num(np64(x)) for x in (cache.k, cache.v))
    vp[pg, :, row] = 0.0
    ro, rl, to, tl = R.decode(np64(q), kp, vp, table, lens, np.array([0, 1]), **weight_parts(fmt, 14))
    if fmt == "mxfp8":
        cache.v_scales[pg, :, row] = 246
    else:
        cache.v[pg, :, row] *= 2.0**120
    o, lse = J.decode(q.cuda(), cache, cu(table), cu(np.array(lens)))
    assert J.device_status() == 0
    assert np.all(np.abs(np64(o) - ro) <= to) and np.all(np.abs(np64(lse) - rl) <= tl)


def test_exponents_that_begin_with_zeros():
    """Units whose first blocks of keys are all of exponent 0, with and without codes, before values of every size."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens, page, H, D = [100, 70, 33], 32, 2, 64
    for shift in (-90, -30, 0, 60):
        for codes in (False, True):
            cache, table, _ = fill_cache(J, lens, page, H, D, "mxfp8", seed=251)
            shift_values(cache, shift)
            for b, p, pg, at in rows_of(table, lens, page):
                if p < 32 or p % 7 == 0:
                    cache.v_scales[pg, :, at] = 0
                    if not codes:
                        cache.v[pg, :, at] = 0
            check_repeated(J, cache, table, lens, [1, 2, 1], 2 * H, 2, spread=14)


@pytest.mark.parametrize("low", [False, True], ids=["level", "beside_small_blocks"])
@pytest.mark.parametrize("code", [0x7f, 0xff])
def test_nan_codes_are_nan_in_v(code, low):
    """E4M3's own NaN, which other writers of a wrapped cache may use: the same in decode, whichever products its keys
    take (blocks far below their neighbours take others), and in cache_read."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens, page, H, D = [90], 32, 2, 128
    cache, table, _ = fill_cache(J, lens, page, H, D, "mxfp8", seed=261)
    at = lambda p: (int(table[0, p // page]), 0, p % page)  # noqa: E731
    if low:
        for p in (64, 80):
            cache.v_scales[at(p)] = 60
    kp, vp = pages_of(cache)
    q = torch.randn(3, H, D, generator=torch.Generator().manual_seed(262)).to(torch.bfloat16)
    q_off = np.array([0, 3])
    ro, rl, to, tl = R.decode(np64(q), kp, vp, table, lens, q_off, causal=True, **weight_parts("mxfp8", 14))
    for p, column in ((88, 7), (89, 100)):  # seen by the last two rows, and by the last
        cache.v[at(p)][column] = code
    o, lse = J.decode(q.cuda(), cache, cu(table), cu(np.array(lens)), q_off=cu(q_off), causal=True)
    assert J.device_status() == 0
    want = np.zeros(ro.shape, bool)
    want[1:, 0, 7] = want[2, 0, 100] = True
    assert np.array_equal(np.isnan(np64(o)), want)
    assert np.all(np.abs(np64(o) - ro)[~want] <= to[~want])
    assert np.all(np.abs(np64(lse) - rl) <= tl)
    _, v = J.cache_read(cache, cu(table), cu(np.array([0, 90])))
    assert torch.isnan(v).nonzero().tolist() == [[88, 0, 7], [89, 0, 100]]


@pytest.mark.parametrize("act", ["softmax", "silu"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["k_nan_block", "k_nan_block_of_zeros", "k_nan_code", "k_large", "v_nan_block", "v_nan_code"])
def test_masked_places_of_an_mxfp8_cache_never_reach_a_row(kind, D, act):
    """NaN blocks (exponent 255, whatever the codes), NaN codes and very large finite keys at the last position: the last
    row, which alone sees it, is NaN (but for the large key), the others are within the bounds of the keys they see."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, page, lens, lq = 2, 16, [50, 21], 4
    q = torch.randn(2 * lq, 2 * H, D, generator=torch.Generator().manual_seed(271)).to(torch.bfloat16)
    q_off = np.array([0, lq, 2 * lq])
    for mask in (dict(causal=True), dict(causal=True, window=5), dict(causal=True, block=49)):
        cache, table, pages = fill_cache(J, lens, page, H, D, "mxfp8", seed=272)
        ro, rl, to, tl = R.decode(np64(q), pages[0], pages[1], table, lens, q_off, act=act, **weight_parts("mxfp8", 14),
                                  **mask)
        for b, n in enumerate(lens):
            at = (int(table[b, (n - 1) // page]), slice(None), (n - 1) % page)
            codes, e = (cache.k, cache.k_scales) if kind[0] == "k" else (cache.v, cache.v_scales)
            if "block" in kind:
                e[at][:, 1] = 255
            if "zeros" in kind or kind == "v_nan_block":
                codes[at][:, 32:64] = 0
            if "code" in kind:
                codes[at][:, 40] = 0x7f
            if kind == "k_large":
                e[at] = 246
        o, lse = J.decode(q.cuda(), cache, cu(table), cu(np.array(lens)), q_off=cu(q_off), act=act, **mask)
        assert J.device_status() == 0
        last = np.zeros(2 * lq, bool)
        last[[lq - 1, 2 * lq - 1]] = True
        got = np64(o)
        assert np.all(np.abs(got - ro)[~last] <= to[~last])
        bad = np.isnan(got[last])
        if kind[0] == "v":
            columns = slice(40, 41) if "code" in kind else slice(32, 64)
            assert bad[..., columns].all()
            bad[..., columns] = False
            assert not bad.any()
        elif kind != "k_large":
            assert bad.all()
        if act == "softmax":
            assert np.all(np.abs(np64(lse) - rl)[~last] <= tl[~last])
            assert kind[0] == "v" or kind == "k_large" or np.isnan(np64(lse)[last]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_keys_of_the_smallest_exponents(D):
    """K blocks of exponents 0 to 3 against query rows of 2^120: scores of ordinary size."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens, page, H = [60, 1, 35], 16, 2
    cache, table, _ = fill_cache(J, lens, page, H, D, "mxfp8", seed=281)
    g = torch.Generator().manual_seed(282)
    cache.k_scales.copy_(torch.randint(0, 4, cache.k_scales.shape, generator=g).to(torch.uint8))
    for b, p, pg, at in rows_of(table, lens, page):
        if p % 3 == 0:
            cache.k_scales[pg, :, at] = 0
    kp, vp = pages_of(cache)
    q = (torch.randn(3, 2 * H, D, generator=g) * 2.0**120).to(torch.bfloat16)
    ro, rl, to, tl = R.decode(np64(q), kp, vp, table, lens, np.arange(4), scale=2.0**-5, **weight_parts("mxfp8"))
    o, lse = J.decode(q.cuda(), cache, cu(table), cu(np.array(lens)), scale=2.0**-5)
    assert J.device_status() == 0
    assert np.all(np.abs(np64(o) - ro) <= to) and np.all(np.abs(np64(lse) - rl) <= tl)
