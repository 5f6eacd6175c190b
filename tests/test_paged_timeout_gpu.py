"""Waits of the paged attention kernels that give up: the call reports it, everything that it has in flight
ends, and with its workspace zeroed the next call is right."""
import pytest
import torch

from mixed_head_causal_b200 import saf
from tests.test_paged_gpu import Cache, pattern

pytestmark = pytest.mark.gpu


@pytest.fixture
def wait_limit():
    yield saf.selftest_serving_wait_limit
    saf.selftest_serving_wait_limit(0)


def calls(B, H, Hkv, T, lens, prefix, mask):
    """A workspace, and a call on it."""
    c = Cache(lens, Hkv, 64, seed=3, prefix=prefix)
    table, seq = c.gpu()
    a, r = (x.cuda() for x in pattern(H, prefix + max(lens), torch.Generator().manual_seed(1)))
    q = torch.randn(B, H, T, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    ws = saf.new_paged_workspace(c.kv, B, H, T, prefix)
    pages = torch.from_numpy(c.prefix_table).cuda()
    kw = dict(alpha=a, rho=r, mask=mask, max_len=max(lens), workspace=ws)

    def call():
        if prefix:
            return saf.paged_attn_prefix(q, c.kv, pages, prefix, table, seq, **kw)
        return saf.paged_attn(q, c.kv, table, seq, **kw)

    return ws, call


@pytest.mark.parametrize("H,Hkv,T,lens,prefix", [
    (4, 4, 1, [9000, 700, 1, 4000], 0),         # the kernel for few rows
    (8, 2, 5, [3000, 700, 5, 4000], 0),         # its form for 20 rows
    (4, 4, 200, [5000, 700, 200, 4000], 0),     # the tensor-core kernel
    (4, 4, 1, [900, 700, 1, 400], 5000),        # two launches for few rows
    (4, 4, 64, [900, 700, 64, 400], 5000),      # two of many
], ids=["decode", "draft", "chunk", "prefix", "prefix_chunk"])
@pytest.mark.parametrize("limit", [1, 300, 3000])
def test_waits_that_give_up(wait_limit, H, Hkv, T, lens, prefix, limit):
    ws, call = calls(4, H, Hkv, T, lens, prefix, [h % 2 for h in range(H)])
    want = [x.clone() for x in call()]
    assert saf.device_status(ws) == saf.SAF_OK
    for _ in range(3):
        wait_limit(limit)
        call()
        call()      # behind one that gave up, its pieces uncounted
        status = saf.device_status(ws)
        # a wait polls once before it looks at the limit, so that a long limit may do; a cycle never does for all of them
        assert status == saf.SAF_ERR_TIMEOUT or (limit > 1 and status == saf.SAF_OK)
        wait_limit(0)
        ws.zero_()
        got = call()
        assert saf.device_status(ws) == saf.SAF_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_limit_refusals():
    for bad in (-1, (1 << 31) + 1):
        with pytest.raises(saf.SafError):
            saf.selftest_serving_wait_limit(bad)


@pytest.mark.parametrize("T", [1, 40])
def test_nothing_waits_for_the_limit(T):
    """Many items to a CTA, whose slots are used again and again: no wait at the end of a CTA looks for a phase that is past."""
    ws, call = calls(900, 4, 4, T, [T + i % 90 for i in range(900)], 33, [0, 1, 0, 0])
    call()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    call()
    end.record()
    end.synchronize()
    assert begin.elapsed_time(end) < 300        # milliseconds; the limit is a second
    assert saf.device_status(ws) == saf.SAF_OK


@pytest.mark.parametrize("H,Hkv", [(4, 4), (28, 1)], ids=["few_rows", "tensor_core"])
def test_the_prefix_may_take_longer_than_the_limit(wait_limit, H, Hkv):
    """Lengths far apart, so that the prefix's replaced rows, each with its own stretch of r, take longer than the
    axis gives them: the CTAs that are through first go on to the sequences' own keys, and wait for the others for a
    few times the limit (25 us; a wait inside either launch is for a few us, an item's end for 15)."""
    B, T, mask, prefix = 128, 1, [int(2 * h >= H) for h in range(H)], 1 << 20
    g = torch.Generator().manual_seed(1)
    lens = [T + int(n) for n in torch.randint(0, 3000, (B,), generator=g)]
    c = Cache(lens, Hkv, 64, seed=3, prefix=640)
    table, seq = c.gpu()
    pages = torch.from_numpy(c.prefix_table).cuda().repeat(prefix // 640 + 1)[:prefix // 64].contiguous()   # the same ten over and over
    a, r = (x.cuda() for x in pattern(H, prefix + max(lens), g))
    q = torch.randn(B, H, T, 64, generator=g).bfloat16().cuda()
    ws = saf.new_paged_workspace(c.kv, B, H, T, prefix)

    def call():
        return saf.paged_attn_prefix(q, c.kv, pages, prefix, table, seq, alpha=a, rho=r, mask=mask, max_len=max(lens), workspace=ws)

    want = [x.clone() for x in call()]
    assert saf.device_status(ws) == saf.SAF_OK
    wait_limit(48_000)
    for _ in range(3):
        got = call()
        assert saf.device_status(ws) == saf.SAF_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
