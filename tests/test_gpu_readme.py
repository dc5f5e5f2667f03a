"""The README's serving example, run as it stands, against the definitions."""
import os
import re

import numpy as np
import pytest
import torch

from tests import paged_ref as R
from tests.dense_ref import rope_tables
from tests.test_gpu_paged import clear, cu, make_table, np64, prefix, weight_parts

pytestmark = pytest.mark.gpu


def test_readme_serving_example():
    """Keys and queries of prompts and new rows are all rotated at their own positions."""
    import jagged_attention_recsys_gdpa_gb300 as J

    readme = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(readme) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
    (example,) = [b for b in blocks if "paged_cache(" in b]
    clear(J)
    H, D, page = 8, 128, 64
    lens = np.array([70, 1, 128])
    B, off = len(lens), prefix(lens)
    g = torch.Generator().manual_seed(311)
    bf16 = lambda n: torch.randn(n, H, D, generator=g).to(torch.bfloat16)  # noqa: E731
    k, v, k_new, v_new, q_new = bf16(int(off[-1])), bf16(int(off[-1])), bf16(B), bf16(B), bf16(B)
    cos, sin, _ = rope_tables(256, D)
    cos, sin = cos.astype(np.float32), sin.astype(np.float32)
    table, n_pages = make_table(lens + 1, page, seed=312)
    names = dict(torch=torch, J=J, n_pages=n_pages, page_table=cu(table), start=cu(np.zeros(B, np.int64)), off=cu(off),
                 kv_lens=cu(lens), k=k.cuda(), v=v.cuda(), k_new=k_new.cuda(), v_new=v_new.cuda(), q_new=q_new.cuda(),
                 cos=cu(cos), sin=cu(sin))
    exec(example, names)
    assert J.device_status() == 0
    # the cache from the definition: every key rotated at its own position
    kp, vp = np.zeros((n_pages, H, page, D)), np.zeros((n_pages, H, page, D))
    for b in range(B):
        rows = torch.cat([k[off[b]:off[b + 1]], k_new[b:b + 1]]).float().numpy()
        rows = R.dequantise(*R.quantise(R.rope_rows(rows, np.arange(lens[b] + 1), cos, sin).astype(np.float64)))
        values = R.dequantise(*R.quantise(np64(torch.cat([v[off[b]:off[b + 1]], v_new[b:b + 1]]))))
        for p in range(lens[b] + 1):
            kp[table[b, p // page], :, p % page], vp[table[b, p // page], :, p % page] = rows[p], values[p]
    # queries: two products and a sum in fp32, then half a step of bf16
    q = np64(q_new)
    c, s = cos[lens][:, None, :].astype(np.float64), sin[lens][:, None, :].astype(np.float64)
    turned = np.stack([q[..., 0::2] * c - q[..., 1::2] * s, q[..., 0::2] * s + q[..., 1::2] * c], -1).reshape(q.shape)
    size = np.stack([np.abs(q[..., 0::2] * c) + np.abs(q[..., 1::2] * s)] * 2, -1).reshape(q.shape) + \
        np.stack([np.abs(q[..., 0::2] * s) + np.abs(q[..., 1::2] * c)] * 2, -1).reshape(q.shape)
    assert np.all(np.abs(np64(names["q_rot"]) - turned) <= 2.0**-8 * np.abs(turned) + 2.0**-22 * size)
    ro, rl, to, tl = R.decode(np64(names["q_rot"]), kp, vp, table, lens + 1, np.arange(B + 1), **weight_parts("mxfp8"))
    assert np.all(np.abs(np64(names["o"]) - ro) <= to) and np.all(np.abs(np64(names["lse"]) - rl) <= tl)
    whole = np.concatenate([R.gather(kp, table, b, lens[b] + 1) for b in range(B)])
    assert np.array_equal(np64(names["k_all"]), np64(torch.from_numpy(whole).to(torch.bfloat16)))
