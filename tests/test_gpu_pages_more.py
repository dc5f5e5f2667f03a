"""The page pool where test_gpu_pages does not reach: large calls in graphs, slots beyond 32 bits, empty batches."""
import numpy as np
import pytest
import torch

from tests import rows_ref as R
from tests.test_gpu_pages import agree, clear, cu, prefix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [6, 1500])
def test_calls_in_two_graphs(B):
    """Two captured steps (assign, give part back) of two pools, replayed at the same time on two streams while lengths change:
    each has scratch of its own."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    page, P = 8, 6
    rng = np.random.default_rng(B)
    n_pages = B * P
    sides = []
    for i in range(2):
        pool, table = J.page_pool(n_pages, page), torch.full((B, P), -1, dtype=torch.int32, device="cuda")
        start, off, keep = (torch.zeros(B + (k == 1), dtype=torch.int64, device="cuda") for k in range(3))
        slots = torch.zeros(B * 10, dtype=torch.int64, device="cuda")

        def step(pool=pool, table=table, start=start, off=off, keep=keep, slots=slots):
            J.page_assign(pool, table, start, off=off, slots=slots)
            J.page_release(pool, table, start + off[1:] - off[:-1], keep=keep)

        step()  # nothing to do: no rows
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        sides.append((pool, table, start, off, keep, slots, graph, torch.cuda.Stream(), R.Pool(n_pages, page),
                      np.full((B, P), -1, np.int32)))
    torch.cuda.synchronize()
    lens = [np.zeros(B, np.int64) for _ in range(2)]
    plans = [[], []]
    for turn in range(8):
        for i in range(2):
            new = np.minimum(rng.integers(0, 11, B), P * page - lens[i])
            kept = rng.integers(0, lens[i] + new + 1)
            plans[i].append((lens[i].copy(), new, kept))
            lens[i] = kept
    inputs = [[(cu(s), cu(prefix(n)), cu(k)) for s, n, k in plan] for plan in plans]
    torch.cuda.synchronize()
    got = [[], []]
    for turn in range(8):
        for i, (pool, table, start, off, keep, slots, graph, stream, ref, t) in enumerate(sides):
            with torch.cuda.stream(stream):
                for to, of in zip((start, off, keep), inputs[i][turn]):
                    to.copy_(of)
                graph.replay()
                got[i].append(slots.clone())
    torch.cuda.synchronize()
    assert J.device_status() == 0
    for i, (pool, table, start, off, keep, slots, graph, stream, ref, t) in enumerate(sides):
        for turn, (s, n, k) in enumerate(plans[i]):
            want = ref.assign(t, s, n, B * 10)
            assert want is not None and np.array_equal(got[i][turn].cpu().numpy(), want)
            assert ref.release(t, s + n, k)
        agree(pool, table, ref, t)


@pytest.mark.parametrize("B", [4, 1100])
def test_slots_beyond_32_bits(B):
    """Pages of 4,096 rows with numbers beyond 2^20."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    n, page, P = 3_000_000, 4096, 3
    free = torch.arange(n, dtype=torch.int32, device="cuda")  # the last page first
    pool, table = J.PagePool(free, cu(np.array([n])), page), torch.full((B, P), -1, dtype=torch.int32, device="cuda")
    lens = np.array([1, 4096, 4097, 9000] * (B // 4))
    slots = J.page_assign(pool, table, cu(np.zeros(B)), off=cu(prefix(lens)))
    ref = R.Pool(1, page)
    ref.free, ref.n = list(range(n)), n
    t = np.full((B, P), -1, np.int32)
    want = ref.assign(t, np.zeros(B, np.int64), lens, int(lens.sum()))
    assert np.array_equal(slots.cpu().numpy(), want) and want.min() > 2**32 and np.array_equal(table.cpu().numpy(), t)
    # a last row inside a page that is there: the others' start would be a page's first row, which takes a page
    inside = (lens - 1) % page != 0
    one = J.page_assign(pool, table, cu(np.where(inside, lens - 1, -1)))
    held = t[np.arange(B), (lens - 1) // page].astype(np.int64) * page + (lens - 1) % page
    assert np.array_equal(one.cpu().numpy(), np.where(inside, held, -1))
    J.page_release(pool, table, cu(lens))
    assert int(pool.count.item()) == n and torch.equal(pool.free_pages, free) and bool((table == -1).all())
    assert J.device_status() == 0


@pytest.mark.parametrize("B", [3, 2000])
def test_batches_without_rows(B):
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    pool, table = J.page_pool(10, 16), torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
    zero = cu(np.zeros(B))
    assert J.page_assign(pool, table, zero, off=cu(np.zeros(B + 1))).shape == (0,)
    assert bool((J.page_assign(pool, table, zero, off=cu(np.zeros(B + 1)), total=9) == -1).all())
    assert bool((J.page_assign(pool, table, zero - 1) == -1).all())  # every sequence skipped
    J.page_release(pool, table, zero)
    J.page_release(pool, table, zero, keep=zero)
    assert int(pool.count.item()) == 10 and bool((table == -1).all())
    assert J.device_status() == 0
