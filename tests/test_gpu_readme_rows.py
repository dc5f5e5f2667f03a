"""The README's examples of the row operators and the page pool, run as they stand."""
import os
import re

import numpy as np
import pytest
import torch

from tests import rows_ref as R

pytestmark = pytest.mark.gpu


def example(word):
    readme = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(readme) as f:
        (code,) = [b for b in re.findall(r"```python\n(.*?)```", f.read(), flags=re.S) if word in b]
    return code


def test_readme_training_example():
    """It runs and gives gradients to the projection and the norms' weights; q is what the definitions give, to the two
    roundings of bf16 on its way (values of a few units, half a step of 2^-8 each, the first one turned: sqrt(2) of it)."""
    import jagged_attention_recsys_gdpa_gb300 as J

    H, D, max_len = 2, 128, 200
    lens = [70, 1, 128]
    off = torch.tensor([0, 70, 71, 199], device="cuda")
    g = torch.Generator().manual_seed(7)
    x = torch.randn(199, 3 * H, D, generator=g).to(torch.bfloat16)
    fused = x.cuda().requires_grad_(True)
    w = [(1 + 0.1 * torch.randn(D, generator=g)).cuda().requires_grad_(True) for _ in range(4)]
    env = dict(J=J, H=H, D=D, max_len=max_len, off=off, fused=fused, wq=w[0], bq=w[1], wk=w[2], bk=w[3])
    exec(example("fused projection"), env)
    env["o"].sum().backward()
    assert J.device_status() == 0
    assert fused.grad.shape == fused.shape and bool(torch.isfinite(fused.grad.float()).all())
    for p in w:
        assert bool(torch.isfinite(p.grad).all())
    assert all(bool((p.grad != 0).any()) for p in (fused, w[0], w[2]))
    v = x[:, :H].double().numpy()
    d = v - v.mean(-1, keepdims=True)
    y = d / np.sqrt((d * d).mean(-1, keepdims=True) + 1e-5) * w[0].detach().cpu().double().numpy() + w[1].detach().cpu().double().numpy()
    theta, size = R.theta(D, 10000.0, "yarn", 4.0, 4096)
    ang = np.concatenate([np.arange(n) for n in lens])[:, None, None] * theta
    a, b, c, s = y[..., :D // 2], y[..., D // 2:], np.cos(ang) * size, np.sin(ang) * size
    want = np.concatenate([a * c - b * s, a * s + b * c], -1)
    length = np.sqrt(a * a + b * b) * size  # of a pair: what its roundings are relative to
    bound = 2.0**-8 * 1.01 * np.concatenate([length, length], -1) * 2 + 1e-6
    assert np.all(np.abs(R.np64(env["q"]) - want) <= bound)


def test_readme_pages_example():
    """New rows get slots of pages of their own, and what is not kept comes back."""
    import jagged_attention_recsys_gdpa_gb300 as J

    page_size, n_pages = 16, 20
    page_table = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
    kv_lens = torch.zeros(3, dtype=torch.int64, device="cuda")
    off = torch.tensor([0, 40, 41, 57], device="cuda")
    new_lens, kept = torch.tensor([40, 1, 16], device="cuda"), torch.tensor([17, 0, 16], device="cuda")
    env = dict(J=J, n_pages=n_pages, page_size=page_size, page_table=page_table, kv_lens=kv_lens, off=off, total=57,
               new_lens=new_lens, kept=kept)
    exec(example("page_assign"), env)
    assert J.device_status() == 0
    assert len(set(env["slots"].tolist())) == 57 and int(env["slots"].min()) >= 0
    assert (page_table >= 0).sum(1).tolist() == [2, 0, 1] and int(env["pool"].count) == n_pages - 3
