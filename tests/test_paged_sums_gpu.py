"""A row's weights sum to one as they are used: where all values of a K/V head are alike, the output is that value.

The weights enter the second product rounded to bf16 (2^-8 of each at most); divided by the sum of the weights before
they are rounded, a row that one key dominates is off by as much.  Divided by the sum of the rounded ones the output is
the value up to fp32 sums (n u32 at the very most, 2000 * 2^-24 = 1.2e-4, under the half step of 2^-9 or more that
would take the bf16 result off), so it is equal.  That holds for replaced rows, as in the layer's forward, and for all
rows of the kernel for few of them; ordinary rows of the tensor-core kernel, as the layer's, are divided by the sum of the
weights: 2^-8 off at most, and 2^-8 again for the result."""
import pytest
import torch

from mixed_head_causal_b200 import saf
from tests.test_paged_gpu import U16, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,T,replaced,prefix,lens", [
    (4, 4, 1, [1, 3], 0, [1, 64, 65, 700, 1999]),
    (8, 2, 2, [1, 3, 4], 0, [2, 64, 65, 700, 1999]),
    (8, 2, 6, [1, 3, 4], 0, [6, 64, 65, 700, 1999]),
    (4, 2, 40, [1, 2, 3], 0, [40, 64, 130, 700, 1999]),
    (4, 2, 200, [1, 2], 0, [200, 300, 513]),
    (4, 2, 1, [2, 3], 777, [3, 90, 1, 64, 200]),
    (4, 4, 1, [1, 2], 500, list(range(1, 1400, 31))),
    (4, 2, 40, [1, 2, 3], 290, [40, 41, 170, 300, 45]),
], ids=["decode", "rows8", "draft", "chunk", "chunk200", "prefix", "prefix_far", "prefix_chunk"])
@pytest.mark.parametrize("scale", [1.0, 4.0])
def test_equal_values_come_out_exactly(H, Hkv, T, replaced, prefix, lens, scale):
    B = len(lens)
    c = Cache(lens, Hkv, 32, seed=H + T, prefix=prefix)
    g = torch.Generator().manual_seed(T)
    value = torch.randn(Hkv, 64, generator=g).bfloat16().cuda()
    c.v.copy_(value[:, None].expand_as(c.v))
    table, seq = c.gpu()
    n = prefix + max(lens)
    a, r = (scale * torch.randn(H, n, generator=g).cuda() for _ in range(2))
    q = scale * torch.randn(B, H, T, 64, generator=g).bfloat16().cuda()
    kw = dict(alpha=a, rho=r, mask=[h in replaced for h in range(H)], max_len=max(lens))
    if prefix:
        o, _ = saf.paged_attn_prefix(q, c.kv, torch.from_numpy(c.prefix_table).cuda(), prefix, table, seq, **kw)
    else:
        o, _ = saf.paged_attn(q, c.kv, table, seq, **kw)
    want = value.repeat_interleave(H // Hkv, 0)[None, :, None].expand_as(o)
    off = (o.double() / want.double() - 1).abs().amax((0, 2, 3))
    few = H // Hkv * T <= 24 and (not prefix or B * H // Hkv * T <= 24)     # (rows of an item, of either launch)
    for h in range(H):
        assert off[h] == 0 if few or h in replaced else off[h] <= (1 + U16) ** 2 - 1, (h, float(off[h]))
