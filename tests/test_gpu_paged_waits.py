"""Decode's bounded waits when they run out while the copies are landing."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import clear, cu, fill_cache

pytestmark = pytest.mark.gpu

TIMEOUT = 6


@pytest.mark.parametrize("Hq,fmt", [(2, "bf16"), (64, "bf16"), (24, "mxfp8")], ids=["one_warp", "two_warps", "tiles"])
def test_a_limit_as_short_as_the_copies_take(Hq, fmt):
    """Limits from far below to above the time that a copy takes: every call ends, one that reports nothing is right, and
    so is the one after."""
    import jagged_attention_recsys_gdpa_gb300 as J
    from jagged_attention_recsys_gdpa_gb300 import _binding as B

    clear(J)
    lens = [4000, 70, 3, 900]
    cache, table, _ = fill_cache(J, lens, 64, 1, 128, fmt, seed=49)
    q = torch.randn(4, Hq, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    args = (q, cache, cu(table), cu(np.array(lens)))
    o, lse = J.decode(*args)
    assert J.device_status() == 0
    try:
        for limit in (1, 300, 600, 1000, 1500, 2000, 3000, 5000, 20000):
            for _ in range(10):
                B.debug_set(0, limit)
                o2, lse2 = J.decode(*args)
                code = J.device_status()
                assert code in (0, TIMEOUT)
                assert code == TIMEOUT or (torch.equal(o, o2) and torch.equal(lse, lse2))
    finally:
        B.debug_set(0, 0)
    o2, lse2 = J.decode(*args)
    assert J.device_status() == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
