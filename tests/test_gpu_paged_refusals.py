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


def test_outputs_that_overlap():
    """Through the Python calls: outputs that share memory with an input or with each other."""
    import jagged_attention_recsys_gdpa_gb300 as J

    cache, table, _ = fill_cache(J, [40, 70], 16, 2, 64, "bf16", seed=302)
    table, kv = cu(table), cu(np.array([40, 70]))
    flat = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = flat[:2]
    for out in (flat[:2], flat[1:]):
        with pytest.raises(J.JattnError):
            J.decode(q, cache, table, kv, out=out)
    with pytest.raises(J.JattnError):
        J.decode(q, cache, table, kv, lse=flat.view(torch.float32).view(-1)[:4].view(2, 2))
    off = cu(np.array([0, 1, 2]))
    with pytest.raises(J.JattnError):
        J.cache_read(cache, table, off, k=flat[:2], v=flat[1:])
    one = J.PagedCache(cache.k, cache.k)  # read only is fine
    J.decode(q, one, table, kv)
    with pytest.raises(J.JattnError):
        J.cache_append(one, flat[:2].clone(), flat[:2].clone(), table, cu(np.array([3, 4])))
    assert J.device_status() == 0


def test_tensors_that_need_a_gradient():
    """None of the operators has a backward pass: buffers and outputs that need a gradient are refused, as q and new rows
    are (outputs under no_grad are written)."""
    import jagged_attention_recsys_gdpa_gb300 as J

    cache, table, _ = fill_cache(J, [40, 70], 16, 2, 64, "bf16", seed=303)
    table, kv, off = cu(table), cu(np.array([40, 70])), cu(np.array([0, 1, 2]))
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    leaf = torch.zeros_like(q).requires_grad_(True)
    lse = torch.zeros(2, 2, device="cuda").requires_grad_(True)
    for kw in (dict(out=leaf), dict(lse=lse)):
        with pytest.raises(ValueError, match="gradient"):
            J.decode(q, cache, table, kv, **kw)
    for kw in (dict(k=leaf), dict(v=leaf)):
        with pytest.raises(ValueError, match="gradient"):
            J.cache_read(cache, table, off, **kw)
    for k, v in ((cache.k.clone().requires_grad_(True), cache.v), (cache.k, cache.v.clone().requires_grad_(True))):
        with pytest.raises(ValueError, match="gradient"):
            J.PagedCache(k, v)
    with torch.no_grad():
        J.decode(q, cache, table, kv, out=leaf, lse=lse)
        J.cache_read(cache, table, off, k=leaf)
    J.PagedCache(cache.k.clone().requires_grad_(True).detach(), cache.v)
    assert J.device_status() == 0
