"""Paged-cache calls that have to be refused, on the GPU."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import OFFSETS, clear, cu, fill_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("B", [60, 400])
def test_offsets_that_name_the_same_rows_again_and_again(B, fmt):
    """Every other sequence claims all query rows: no batch of prefix sums has that much work. Nothing is written, and the
    next call is right."""
    import jagged_attention_recsys_gdpa_gb300 as J

    clear(J)
    lens = [300] * B
    cache, table, _ = fill_cache(J, lens[:1], 64, 1, 64, fmt, seed=301)
    table = cu(np.tile(table, (B, 1)))
    q = torch.randn(B, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    kv = cu(np.array(lens))
    good = J.decode(q, cache, table, kv)
    assert J.device_status() == 0
    off = np.zeros(B + 1, np.int64)
    off[1::2] = B
    off[-1] = B
    out, lse = torch.full_like(q, 5.0), torch.full((B, 4), 5.0, device="cuda")
    J.decode(q, cache, table, kv, q_off=cu(off), out=out, lse=lse)
    assert J.device_status() == OFFSETS
    assert bool((out == 5.0).all()) and bool((lse == 5.0).all())
    o, l2 = J.decode(q, cache, table, kv, q_off=cu(np.arange(B + 1)))
    assert J.device_status() == 0 and torch.equal(o, good[0]) and torch.equal(l2, good[1])
