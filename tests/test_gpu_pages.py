"""The page pool on the GPU against a pool kept as a list, and the operators
between projections and attention used together: training through norm, rotation
and jagged attention, and serving through norm, rotation, pages, cache and decode."""
import numpy as np
import pytest
import torch

from tests import paged_ref as P
from tests import rows_ref as R
from tests.dense_ref import dense_forward
from tests.rows_ref import np64

pytestmark = pytest.mark.gpu

OFFSETS, PAGES, LENGTH, POOL = 5, 10, 11, 12


def cu(x, dtype=np.int64):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).cuda()


def prefix(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def clear(J):
    J.device_status()
    J.device_status()


def agree(pool, table, ref, ref_table):
    n = int(pool.count.item())
    assert n == len(ref.free)
    assert pool.free_pages[:n].tolist() == ref.free
    assert np.array_equal(table.cpu().numpy(), ref_table)


# the last two are past what one CTA serves
@pytest.mark.parametrize("B,P_,page,most", [(1, 3, 8, 5), (5, 7, 16, 40), (64, 9, 1, 3), (33, 20, 4096, 9000), (1024, 4, 32, 4),
                                            (7, 300, 16, 2000), (1025, 6, 8, 20), (700, 40, 64, 1200)])
def test_pages_come_and_go(B, P_, page, most):
    """Sequences that grow by random amounts, shrink and leave, many times, against the list."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    rng = np.random.default_rng(B)
    n_pages = B * P_ // 2 + 3
    pool, ref = J.page_pool(n_pages, page), R.Pool(n_pages, page)
    ref_table = np.full((B, P_), -1, np.int32)
    table = torch.from_numpy(ref_table.copy()).cuda()
    lens = np.zeros(B, np.int64)
    for turn in range(12):
        new = rng.integers(0, most + 1, B) * (rng.random(B) < 0.7)
        new = np.minimum(new, P_ * page - lens)
        start = np.where(rng.random(B) < 0.1, -1 - lens, lens)  # some sequences are not in the batch
        off = prefix(new)
        total = int(off[-1]) + int(rng.integers(0, 4))  # a padded batch
        want = ref.assign(ref_table, start, new, total)
        slots = J.page_assign(pool, table, cu(start), off=cu(off), total=total)
        if want is None:  # the pool is short: nothing moved
            assert J.device_status() == POOL and bool((slots == -1).all())
            agree(pool, table, ref, ref_table)
        else:
            assert J.device_status() == 0
            assert np.array_equal(slots.cpu().numpy(), want)
            lens = lens + np.where(start >= 0, new, 0)
            agree(pool, table, ref, ref_table)
        kind = rng.random(B)
        keep = np.where(kind < 0.3, 0, np.where(kind < 0.6, lens, np.where(kind < 0.7, -1, rng.integers(0, lens + 1))))
        assert ref.release(ref_table, lens, keep)
        J.page_release(pool, table, cu(lens), keep=cu(keep))
        assert J.device_status() == 0
        agree(pool, table, ref, ref_table)
        lens = np.where(keep < 0, lens, keep)
    # one row each, without offsets
    start = np.minimum(lens, P_ * page - 1)
    lens = start + 1
    want = ref.assign(ref_table, start, np.ones(B, np.int64), B)
    slots = J.page_assign(pool, table, cu(start))
    if want is not None:
        assert np.array_equal(slots.cpu().numpy(), want)
        agree(pool, table, ref, ref_table)
        ref.release(ref_table, lens, None)
        J.page_release(pool, table, cu(lens))
        agree(pool, table, ref, ref_table)
    J.device_status()


@pytest.mark.parametrize("B", [3, 1500])
def test_page_errors_leave_everything_else_alone(B):
    """Each in a call that one CTA serves and in a large one."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    page, P_ = 8, 4

    def fresh():
        pool, ref = J.page_pool(B * 3, page), R.Pool(B * 3, page)
        t = np.full((B, P_), -1, np.int32)
        return pool, torch.from_numpy(t.copy()).cuda(), ref, t

    ten = np.full(B, 10, np.int64)
    zero = np.zeros(B, np.int64)
    # lengths past the table: that sequence alone goes without
    for start in (25, 33, 2**40, 2**62):
        pool, table, ref, t = fresh()
        s = zero.copy()
        s[1] = start
        want = ref.assign(t, s, ten, 10 * B)
        slots = J.page_assign(pool, table, cu(s), off=cu(prefix(ten)))
        assert J.device_status() == LENGTH and np.array_equal(slots.cpu().numpy(), want)
        assert bool((slots[10:20] == -1).all()) and bool((slots[:10] >= 0).all())
        agree(pool, table, ref, t)
    # offsets that are no prefix sums: whatever they claim, each slot is one of a page of the pool, or -1
    for at, value in ((1, 10 * B + 1), (2, 5), (0, 3), (0, -2), (B, 10 * B + 5), (1, -7), (1, 2**62), (2, -2**62)):
        pool, table, ref, t = fresh()
        off = prefix(ten)
        off[at] = value
        slots = J.page_assign(pool, table, cu(zero), off=cu(off), total=10 * B)
        assert J.device_status() in (OFFSETS, LENGTH, POOL), (at, value)
        assert bool(((slots >= -1) & (slots < 3 * B * page)).all())
        assert bool(((table >= -1) & (table < 3 * B)).all())
        taken = table[table >= 0]
        assert len(set(taken.tolist())) == taken.numel() == 3 * B - int(pool.count.item())
    # a pool that is short, or whose height is none
    for count in (0, 2 * B - 1, -1, 3 * B + 1, 2**40):
        pool, table, ref, t = fresh()
        pool.count.fill_(count)
        slots = J.page_assign(pool, table, cu(zero), off=cu(prefix(ten)))
        assert J.device_status() == POOL and bool((slots == -1).all()) and bool((table == -1).all())
        assert int(pool.count.item()) == count
    # numbers on the stack, or in the table, that are no pages
    pool, table, ref, t = fresh()
    pool.free_pages[-1] = 3 * B
    slots = J.page_assign(pool, table, cu(zero), off=cu(prefix(ten)))
    assert J.device_status() == PAGES
    assert bool((slots[:8] == -1).all()) and int(table[0, 0]) == -1 and bool((slots[8:] >= 0).all())
    pool, table, ref, t = fresh()
    ref.assign(t, zero, ten, 10 * B)
    J.page_assign(pool, table, cu(zero), off=cu(prefix(ten)), slots=False)
    for bad in (-1, 3 * B, 2**31 - 1):
        pool2, table2 = J.PagePool(pool.free_pages.clone(), pool.count.clone(), page), table.clone()
        ref2, t2 = R.Pool(3 * B, page), t.copy()
        ref2.free = list(ref.free)
        table2[2, 1] = t2[2, 1] = bad
        slots = J.page_assign(pool2, table2, cu(ten))  # the row behind the tenth lies in that page
        assert J.device_status() == PAGES and int(slots[2]) == -1 and int(slots[0]) == int(t[0, 1]) * 8 + 2
        J.page_release(pool2, table2, cu(ten))
        assert J.device_status() == PAGES
        ref2.release(t2, ten, None)
        agree(pool2, table2, ref2, t2)
        assert int(table2[2, 0]) == int(t[2, 0])  # it keeps all it has
    # lengths past the table, and pages given back to a full pool
    for n in (33, 2**40, 2**62):
        pool2, table2 = J.PagePool(pool.free_pages.clone(), pool.count.clone(), page), table.clone()
        ref2, t2 = R.Pool(3 * B, page), t.copy()
        ref2.free = list(ref.free)
        lens = ten.copy()
        lens[0] = n
        J.page_release(pool2, table2, cu(lens))
        assert J.device_status() == LENGTH
        ref2.release(t2, lens, None)
        agree(pool2, table2, ref2, t2)
    for count in (3 * B - 2 * B + 1, 3 * B, -1, 3 * B + 7):
        pool2, table2 = J.PagePool(pool.free_pages.clone(), pool.count.clone(), page), table.clone()
        pool2.count.fill_(count)
        before = pool2.free_pages.clone()
        J.page_release(pool2, table2, cu(ten))
        assert J.device_status() == POOL
        assert torch.equal(table2, table) and torch.equal(pool2.free_pages, before) and int(pool2.count.item()) == count
    J.page_release(pool, table, cu(ten), keep=cu(np.full(B, 10)))  # nothing to give
    J.page_release(pool, table, cu(ten), keep=cu(np.full(B, 12)))
    J.page_release(pool, table, cu(np.full(B, -4)))
    assert J.device_status() == 0 and np.array_equal(table.cpu().numpy(), t)


@pytest.mark.parametrize("B", [3, 900])
@pytest.mark.parametrize("rows", [1, 3, 4, 5, 8, 9])
def test_page_errors_of_a_few_rows_each(B, rows):
    """Calls whose sequences move no more pages than a thread holds, and one more: sequences past their table, bad offsets, short
    pools, numbers that are no pages, padding, each against the list or in what it may touch."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    page, P_ = 2, 7
    n_pages = B * 7
    new = np.full(B, rows, np.int64)
    total = B * rows + 3
    for first in (0, 1, 2, 5):
        pool, ref = J.page_pool(n_pages, page), R.Pool(n_pages, page)
        t = np.full((B, P_), -1, np.int32)
        before = np.full(B, first, np.int64)
        assert ref.assign(t, np.zeros(B, np.int64), before, first * B) is not None
        table = torch.from_numpy(np.full((B, P_), -1, np.int32)).cuda()
        J.page_assign(pool, table, cu(np.zeros(B)), off=cu(prefix(before)))
        agree(pool, table, ref, t)

        def copies():
            p2, r2 = J.PagePool(pool.free_pages.clone(), pool.count.clone(), page), R.Pool(n_pages, page)
            r2.free = list(ref.free)
            return p2, table.clone(), r2, t.copy()

        # rows behind the table, sequences that are skipped
        p2, table2, r2, t2 = copies()
        start = before.copy()
        start[1], start[2] = 2**40, -5
        want = r2.assign(t2, start, new, total)
        slots = J.page_assign(p2, table2, cu(start), off=cu(prefix(new)), total=total)
        assert J.device_status() == LENGTH and np.array_equal(slots.cpu().numpy(), want)
        agree(p2, table2, r2, t2)
        # without slots, and given back: all as before
        p2, table2, r2, t2 = copies()
        assert J.page_assign(p2, table2, cu(before), off=cu(prefix(new)), total=total, slots=False) is None
        assert r2.assign(t2, before, new, total) is not None
        agree(p2, table2, r2, t2)
        J.page_release(p2, table2, cu(before + rows), keep=cu(before))
        assert J.device_status() == 0
        agree(p2, table2, ref, t)
        # offsets that are no prefix sums
        for at, value in ((1, total + 9), (2, 0), (0, 1), (0, -2), (B, total + 5), (1, -7), (1, 2**62), (2, -2**62)):
            p2, table2, r2, t2 = copies()
            off = prefix(new)
            off[at] = value
            slots = J.page_assign(p2, table2, cu(before), off=cu(off), total=total)
            assert J.device_status() in (OFFSETS, LENGTH, POOL), (at, value)
            assert bool(((slots >= -1) & (slots < n_pages * page)).all())
            taken = table2[table2 >= 0]
            assert len(set(taken.tolist())) == taken.numel() == n_pages - int(p2.count.item())
        # a pool without enough
        p2, table2, r2, t2 = copies()
        need = int((-(-(first + rows) // page) - (-(-first // page))) * B)
        if need > 0:
            p2.count.fill_(need - 1)
            slots = J.page_assign(p2, table2, cu(before), off=cu(prefix(new)), total=total)
            assert J.device_status() == POOL and bool((slots == -1).all()) and torch.equal(table2, table)
            assert int(p2.count.item()) == need - 1
            # a number that is no page on top of the stack: the first sequence's first page
            p2, table2, r2, t2 = copies()
            good = p2.free_pages.clone()
            p2.free_pages[len(r2.free) - 1] = -3
            slots = J.page_assign(p2, table2, cu(before), off=cu(prefix(new)), total=total)
            assert J.device_status() == PAGES
            p3 = J.PagePool(good, pool.count.clone(), page)
            table3 = table.clone()
            all_good = J.page_assign(p3, table3, cu(before), off=cu(prefix(new)), total=total)
            at = -(-first // page)
            bad = all_good == -2  # none
            lo = max(0, at * page - first)
            bad[lo:min(rows, lo + page)] = True
            assert bool((slots[bad] == -1).all()) and torch.equal(slots[~bad], all_good[~bad])
            table3[0, at] = -1
            assert torch.equal(table2, table3)
    assert J.device_status() == 0


def test_pages_in_graphs_and_on_streams():
    """A captured serving step (pages, append, decode) replayed while lengths grow, and two pools on two streams."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    B, H, D, page, cap = 5, 2, 64, 8, 64
    sides = []
    for i in range(2):
        cache, pool = J.paged_cache(B * cap // page, page, H, D), J.page_pool(B * cap // page, page)
        table = torch.full((B, cap // page), -1, dtype=torch.int32, device="cuda")
        lens = torch.zeros(B, dtype=torch.int64, device="cuda")
        x = torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda")
        slots = torch.zeros(B, dtype=torch.int64, device="cuda")
        out = torch.zeros_like(x)

        def step(cache=cache, pool=pool, table=table, lens=lens, x=x, slots=slots, out=out):
            J.page_assign(pool, table, lens, slots=slots)
            J.cache_append(cache, x, x, table, lens)
            lens.add_(1)
            J.decode(x, cache, table, lens, out=out)

        step()
        J.page_release(pool, table, lens)
        lens.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        sides.append((cache, pool, table, lens, x, slots, out, graph, torch.cuda.Stream()))
    torch.cuda.synchronize()
    rows = [[torch.randn(B, H, D, generator=torch.Generator().manual_seed(100 * i + t)).to(torch.bfloat16) for t in range(30)]
            for i in range(2)]
    got = [[], []]
    for t in range(30):
        for i, (cache, pool, table, lens, x, slots, out, graph, st) in enumerate(sides):
            with torch.cuda.stream(st):
                x.copy_(rows[i][t])
                graph.replay()
                got[i].append(slots.clone())
    torch.cuda.synchronize()
    assert J.device_status() == 0
    for i, (cache, pool, table, lens, x, slots, out, graph, st) in enumerate(sides):
        k, v = J.cache_read(cache, table, cu(prefix([30] * B)))
        want = torch.stack(rows[i], 1).reshape(B * 30, H, D)
        assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
        # the slots name the rows: pages lie [page, head, row]
        flat = cache.k.transpose(1, 2).reshape(-1, H, D)
        assert torch.equal(flat[torch.stack(got[i], 1).reshape(-1)], k)
        assert int(pool.count.item()) == B * cap // page - B * 4
        J.page_release(pool, table, lens)
        assert int(pool.count.item()) == B * cap // page and bool((table == -1).all())


def test_many_rows_of_slots():
    """Whole histories at once: slots against the table on the GPU, no page twice."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    B, page = 3000, 64
    g = torch.Generator().manual_seed(3)
    lens = (torch.rand(B, generator=g) ** 4 * 20_000).long().cuda()
    start = torch.randint(0, 300, (B,), generator=g).cuda()
    off = torch.cat([lens.new_zeros(1), lens.cumsum(0)])
    need, have = (start + lens + page - 1) // page, (start + page - 1) // page
    n = int(need.sum())
    pool = J.page_pool(n, page)
    table = torch.full((B, int(need.max())), -1, dtype=torch.int32, device="cuda")
    first = J.page_assign(pool, table, torch.zeros_like(start), off=torch.cat([start.new_zeros(1), start.cumsum(0)]))
    slots = J.page_assign(pool, table, start, off=off)
    assert J.device_status() == 0 and int(pool.count.item()) == 0
    used = table[torch.arange(table.shape[1], device="cuda")[None] < need[:, None]]
    assert torch.equal(used.sort().values, torch.arange(n, dtype=torch.int32, device="cuda"))
    for s, at, o in ((first, torch.zeros_like(start), torch.cat([start.new_zeros(1), start.cumsum(0)])), (slots, start, off)):
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), o[1:] - o[:-1])
        pos = torch.arange(len(b), device="cuda") - o[b] + at[b]
        assert torch.equal(s, table[b, pos // page].long() * page + pos % page)
    whole = J.page_release(pool, table, start + lens)
    assert whole is None and int(pool.count.item()) == n and bool((table == -1).all())
    assert torch.equal(pool.free_pages.sort().values, torch.arange(n, dtype=torch.int32, device="cuda"))


def test_page_python_refusals():
    import jagged_attention_recsys_gdpa_gb300 as J

    pool = J.page_pool(10, 16)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int64, device="cuda")
    off = torch.tensor([0, 1, 3], device="cuda")
    J.page_assign(pool, table, lens, off=off)
    for kw in (dict(table=table.long()), dict(table=table[:, :2]), dict(table=table[0]), dict(table=table.cpu()), dict(start=lens.int()),
               dict(start=lens[:1]), dict(start=lens.cpu()), dict(off=lens), dict(off=off.int()), dict(off=None, total=3),
               dict(slots=lens.int(), off=None), dict(slots=off), dict(slots=off[:2], total=3)):
        kw = dict(dict(table=table, start=lens, off=off), **kw)
        if kw.get("slots") is off:
            kw["slots"] = off.cpu()
        with pytest.raises(ValueError):
            J.page_assign(pool, kw.pop("table"), kw.pop("start"), **kw)
    for kw in (dict(lens=lens.int()), dict(lens=off), dict(keep=lens.int()), dict(keep=off), dict(table=table.t())):
        kw = dict(dict(table=table, lens=lens, keep=None), **kw)
        with pytest.raises(ValueError):
            J.page_release(pool, kw["table"], kw["lens"], keep=kw["keep"])
    free, count = pool.free_pages, pool.count
    for args in ((free.long(), count, 16), (free[None], count, 16), (free[::2], count, 16), (free[:0], count, 16), (free, count.int(), 16),
                 (free, count[0], 16), (free, count.cpu(), 16), (free, count, 24), (free, count, 0), (free, count, 8192)):
        with pytest.raises(ValueError):
            J.PagePool(*args)
    with pytest.raises(J.JattnError):  # a pool whose height lies on its own stack
        bad = torch.zeros(12, dtype=torch.int32, device="cuda")
        J.page_assign(J.PagePool(bad, bad[2:4].view(torch.int64), 16), table, lens, off=off)
    assert J.device_status() == 0


# ------------------------------------------------------------------ together
def test_training_through_norm_rotation_and_attention():
    """q and k normalised per head, rotated (half layout, half of the columns) and attended over, forward and backward: against the
    same chain in 64 bits by autograd. Values pass bf16 four times on the way (2^-8 each, relative, on numbers of size one), the
    attention's own tolerance is 1e-2 + 1e-2 |ref|; the weights' gradients sum 219 x 2 rows of such errors, which are
    independent: within 1e-2 of the largest of all."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    H, D, lens = 2, 64, [70, 1, 130, 18]
    off = prefix(lens)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(int(off[-1]), 3 * H, D, generator=g).to(torch.bfloat16)
    dy = torch.randn(int(off[-1]), H, D, generator=g).to(torch.bfloat16)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).float() for _ in range(2)]
    b = [(0.2 * torch.randn(D, generator=g)).float() for _ in range(2)]
    o_gpu = cu(off)
    leaf = x.cuda().requires_grad_(True)
    ws, bs = ([t.cuda().requires_grad_(True) for t in v] for v in (w, b))
    tables = J.rotary_tables(140, D // 2)
    q = J.rotary(J.layer_norm(leaf[:, :H], ws[0], bs[0]), tables, off=o_gpu, layout="half")
    k = J.rotary(J.layer_norm(leaf[:, H:2 * H], ws[1], bs[1]), tables, off=o_gpu, layout="half")
    o = J.attention(q, k, leaf[:, 2 * H:].contiguous(), o_gpu, o_gpu, causal=True)
    o.backward(dy.cuda())
    assert J.device_status() == 0

    ref = x.double().requires_grad_(True)
    rw, rb = ([t.double().requires_grad_(True) for t in v] for v in (w, b))
    theta, _ = R.theta(D // 2, 10000.0)
    pos = torch.cat([torch.arange(n) for n in lens]).double()
    c, s = ((f(pos[:, None] * torch.from_numpy(theta)))[:, None] for f in (torch.cos, torch.sin))

    def turned(z):
        a, e = z[..., :16], z[..., 16:32]
        return torch.cat([a * c - e * s, a * s + e * c, z[..., 32:]], -1)

    norm = lambda z, i: torch.nn.functional.layer_norm(z, (D,), rw[i], rb[i], 1e-5)  # noqa: E731
    ro, _ = dense_forward(turned(norm(ref[:, :H], 0)), turned(norm(ref[:, H:2 * H], 1)), ref[:, 2 * H:], off, off, 0, 1, 0, D**-0.5, False)
    ro.backward(dy.double())
    got, want = np64(o), ro.detach().numpy()
    assert np.all(np.abs(got - want) <= 1e-2 + 1e-2 * np.abs(want) + 4 * 2.0**-8)
    got, want = np64(leaf.grad), ref.grad.numpy()
    assert np.all(np.abs(got - want) <= 1e-2 + 1e-2 * np.abs(want) + 4 * 2.0**-8 * np.abs(want).max())
    for i in range(2):
        for a, r in ((ws[i], rw[i]), (bs[i], rb[i])):
            want = r.grad.numpy()
            # biases of keys move all of a query's scores alike: theirs is nearly zero, so the bound goes by the queries' size
            size = max(np.abs(rw[0].grad.numpy()).max(), np.abs(want).max())
            assert np.all(np.abs(np64(a.grad) - want) <= 2e-2 * size)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_serving_through_norm_rotation_pages_and_cache(fmt):
    """Prompts, then single events with drafts that are taken back, users leaving and others coming: queries and keys come out
    of one fused projection, normalised and rotated in place of any copy, and decode agrees with its definition over what
    the cache holds."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    Hq, H, D, page, B, P_ = 4, 2, 64, 16, 4, 12
    n_pages = 30
    cache, pool = J.paged_cache(n_pages, page, H, D, format=fmt), J.page_pool(n_pages, page)
    table = torch.full((B, P_), -1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    w, b = 1 + 0.1 * torch.randn(D, generator=g, device="cuda"), 0.1 * torch.randn(D, generator=g, device="cuda")
    tables = J.rotary_tables(256, D, scaling="yarn", factor=4.0, original=64)
    lens = np.zeros(B, np.int64)
    keys = [[] for _ in range(B)]

    def event(new):
        """new rows of each sequence: pages, projections, norm, rotation, append, decode"""
        nonlocal lens
        off, start = cu(prefix(new)), cu(lens)
        total = int(new.sum())
        slots = J.page_assign(pool, table, start, off=off, total=total)
        fused = torch.randn(total, Hq + 2 * H, D, generator=g, device="cuda").to(torch.bfloat16)
        qk = fused[:, :Hq + H]
        J.layer_norm_forward(qk, w, b, out=qk)
        J.rotary(qk, tables, off=off, start=start, layout="half", out=qk)
        k, v = fused[:, Hq:Hq + H].contiguous(), fused[:, Hq + H:].contiguous()
        J.cache_append(cache, k, v, table, start, off=off)
        lens = lens + new
        for s in range(B):
            keys[s] += [(k[r], v[r], int(slots[r])) for r in range(int(off[s]), int(off[s + 1]))]
        q = fused[:, :Hq].contiguous()
        o, lse = J.decode(q, cache, table, cu(lens), q_off=off, causal=True)
        assert J.device_status() == 0
        if fmt == "bf16":
            pages = [np64(cache.k), np64(cache.v)]
            ref = dict()
        else:
            pages = [P.dequantise(c.cpu().numpy(), e.cpu().numpy()) for c, e in ((cache.k, cache.k_scales), (cache.v, cache.v_scales))]
            ref = dict(part=2.0**-11, floor=2.0**-18)
        ro, rl, to, tl = P.decode(np64(q), *pages, table.cpu().numpy(), lens, prefix(new), causal=True, **ref)
        assert np.all(np.abs(np64(o) - ro) <= to) and np.all(np.abs(np64(lse) - rl) <= tl)

    event(np.array([40, 1, 17, 0]))
    for t in range(4):
        event(np.array([1, 1, 3, 1]))
        back = np.array([0, 0, 2, 0])  # two drafts are not taken
        J.page_release(pool, table, cu(lens), keep=cu(lens - back))
        lens = lens - back
        keys[2] = keys[2][:int(lens[2])]
    keep = lens.copy()
    keep[0] = 0  # the first user leaves and another comes
    J.page_release(pool, table, cu(lens), keep=cu(keep))
    lens, keys[0] = keep, []
    event(np.array([70, 1, 1, 1]))
    # every row is where its slot says, the pages in use and the free ones are all there are
    if fmt == "bf16":
        flat_k, flat_v = (x.transpose(1, 2).reshape(-1, H, D) for x in (cache.k, cache.v))
        for s in range(B):
            for k, v, slot in keys[s]:
                assert torch.equal(flat_k[slot], k) and torch.equal(flat_v[slot], v)
    used = table[table >= 0].tolist() + pool.free_pages[:int(pool.count.item())].tolist()
    assert sorted(used) == list(range(n_pages))
