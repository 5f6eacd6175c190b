"""The README's serving lines, run as they stand."""
import os
import re

import numpy as np
import pytest
import torch

from tests import paged_oracle as O
from tests.test_paged_gpu import check, np64

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("T", [64, 1000, 65])
def test_serving_step(T):
    """With contexts of a multiple of the page size and not, and a table with columns to spare."""
    code = re.search(r"## Serving.*?```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S).group(1)
    B, H = 2, 12
    g = torch.Generator().manual_seed(T)
    lens = [T, T - 17]
    cols = -(-T // 64) + 2
    q, k, v = (torch.randn(B, H, 1, 64, generator=g).bfloat16().cuda() for _ in range(3))
    alpha, rho = (0.5 * torch.randn(H, T, generator=g) for _ in range(2))
    mask = [h in (1, 5) for h in range(H)]
    table = torch.randperm(1024, generator=g)[:B * cols].to(torch.int32).view(B, cols)
    env = dict(T=T, B=B, H=H, mask=mask, q=q, k=k, v=v, alpha=alpha.cuda(), rho=rho.cuda(), table=table.cuda(),
               seq=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    setup, step = code.split("# one decode step", 1)
    exec("import torch\nfrom mixed_head_causal_b200 import saf\n" + setup, env)
    for cache in (env["kv"].k_cache, env["kv"].v_cache):     # the tokens that are cached already
        cache.copy_(torch.randn(cache.shape, generator=g).bfloat16())
    exec("# one decode step" + step, env)
    torch.cuda.synchronize()
    kc, vc = np64(env["kv"].k_cache), np64(env["kv"].v_cache)
    ref = O.attend(np64(env["q1"]), kc, vc, table.numpy(), lens, None, np64(alpha), np64(rho), mask, T)
    check(env["o"], env["lse"], ref, None, 1)
