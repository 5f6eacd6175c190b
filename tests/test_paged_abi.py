"""Refusals of the serving entry points, on the host: every call here fails
its argument checks (or is empty) before anything is enqueued."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from mixed_head_causal_b200 import build as saf_build
from mixed_head_causal_b200 import saf

FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    saf_build.build()
    return saf.load()


def kv(**kw):
    f = dict(k=FAKE, v=FAKE, k_stride_page=4096, k_stride_head=2048, k_stride_slot=64, v_stride_page=4096,
             v_stride_head=2048, v_stride_slot=64, num_pages=8, page_size=32, H_kv=2, d_h=64)
    f.update(kw)
    return saf._PagedKVStruct(*(f[n] for n, _ in saf._PagedKVStruct._fields_))


def strides(*x):
    return (ctypes.c_int64 * 3)(*x)


def append(lib, cache=None, B=2, H=4, T=1, **kw):
    f = dict(q=FAKE, qs=strides(256, 64, 64), k=FAKE, ks=strides(128, 64, 64), v=FAKE, vs=strides(128, 64, 64),
             q_out=FAKE, k_out=None, rope=FAKE, rope_len=64, rot=64, inter=0, off=0, mask=None, table=FAKE, max_pages=2,
             seq=FAKE, ql=None, max_len=64)
    f.update(kw)
    c = cache if cache is not None else kv()
    return lib.saf_kv_append(ctypes.addressof(c), f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["q_out"],
                             f["k_out"], f["rope"], f["rope_len"], f["rot"], f["inter"], f["off"], f["mask"], f["table"],
                             f["max_pages"], f["seq"], f["ql"], B, H, T, f["max_len"], None)


def attn(lib, cache=None, B=2, H=4, T=1, prefix=False, **kw):
    f = dict(q=FAKE, o=FAKE, lse=FAKE, a=FAKE, r=FAKE, plen=128, mask=bytes([0, 1, 0, 0]), ptab=FAKE, pre=40, table=FAKE,
             max_pages=2, seq=FAKE, ql=None, max_len=64, ws=FAKE, wsb=None)
    f.update(kw)
    c = cache if cache is not None else kv()
    wsb = f["wsb"] if f["wsb"] is not None else lib.saf_paged_workspace_size(B, H, 2, T, 40)
    head = [ctypes.addressof(c), f["q"], f["o"], f["lse"], f["a"], f["r"], f["plen"], f["mask"]]
    tail = [f["table"], f["max_pages"], f["seq"], f["ql"], B, H, T, f["max_len"], f["ws"], wsb, None]
    if prefix:
        return lib.saf_paged_attn_prefix(*head, f["ptab"], f["pre"], *tail)
    return lib.saf_paged_attn(*head, *tail)


@pytest.mark.parametrize("call", [append, attn], ids=["append", "attn"])
def test_cache_refusals(lib, call):
    bad, uns = saf.SAF_ERR_INVALID_ARG, saf.SAF_ERR_UNSUPPORTED
    for want, kw in [(uns, dict(d_h=128)), (uns, dict(page_size=8)), (uns, dict(page_size=48)), (uns, dict(page_size=512)),
                     (bad, dict(num_pages=-1)), (bad, dict(H_kv=3)), (bad, dict(H_kv=0)), (bad, dict(H_kv=8)),
                     (bad, dict(k=None)), (bad, dict(v=FAKE + 8)), (bad, dict(k_stride_slot=60)),
                     (bad, dict(v_stride_head=56)), (bad, dict(k_stride_page=-4096)), (bad, dict(v_stride_page=1 << 40))]:
        assert call(lib, cache=kv(**kw)) == want, kw


@pytest.mark.parametrize("call", [append, attn], ids=["append", "attn"])
def test_table_refusals(lib, call):
    bad = saf.SAF_ERR_INVALID_ARG
    for kw in [dict(table=None), dict(seq=None), dict(max_pages=-1), dict(max_len=65), dict(max_len=-1), dict(B=-1), dict(T=-1),
               dict(q=None), dict(q=FAKE + 2), dict(table=FAKE + 2), dict(seq=FAKE + 1), dict(ql=FAKE + 2)]:
        assert call(lib, **kw) == bad, kw
    assert call(lib, H=300, cache=kv(H_kv=300)) == saf.SAF_ERR_UNSUPPORTED


def test_append_refusals(lib):
    bad = saf.SAF_ERR_INVALID_ARG
    for kw in [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(q_out=None), dict(q_out=FAKE + 2), dict(k_out=FAKE + 4),
               dict(rope_len=63), dict(off=1), dict(off=-1), dict(rope=FAKE + 4), dict(ks=strides(128, 60, 64)),
               dict(vs=None), dict(qs=strides(-256, 64, 64))]:
        assert append(lib, **kw) == bad, kw
    for rot in (0, 8, 24, 80, 128):
        assert append(lib, rot=rot, rope_len=1 << 20) == saf.SAF_ERR_UNSUPPORTED
    assert append(lib, B=1 << 20, T=1 << 15) == bad     # more rows than a launch holds


def test_rope_table_refusals(lib):
    assert lib.saf_rope_table(FAKE, 4, 24, 10000.0, None) == saf.SAF_ERR_UNSUPPORTED
    assert lib.saf_rope_table(FAKE, 4, 128, 10000.0, None) == saf.SAF_ERR_UNSUPPORTED
    assert lib.saf_rope_table(FAKE, -1, 64, 10000.0, None) == saf.SAF_ERR_INVALID_ARG
    assert lib.saf_rope_table(FAKE, 4, 64, 0.0, None) == saf.SAF_ERR_INVALID_ARG
    assert lib.saf_rope_table(FAKE, 4, 64, float("nan"), None) == saf.SAF_ERR_INVALID_ARG
    assert lib.saf_rope_table(None, 4, 64, 10000.0, None) == saf.SAF_ERR_INVALID_ARG
    assert lib.saf_rope_table(None, 0, 64, 10000.0, None) == saf.SAF_OK


def test_attention_refusals(lib):
    bad = saf.SAF_ERR_INVALID_ARG
    for kw in [dict(o=None), dict(lse=None), dict(o=FAKE + 2), dict(a=None), dict(r=None), dict(a=FAKE + 4), dict(plen=63)]:
        assert attn(lib, **kw) == bad, kw
    for kw in [dict(ptab=None), dict(ptab=FAKE + 2), dict(pre=-1), dict(plen=103)]:
        assert attn(lib, prefix=True, **kw) == bad, kw
    assert attn(lib, ws=None) == saf.SAF_ERR_WORKSPACE
    assert attn(lib, wsb=saf.paged_workspace_size(2, 4, 1, 2) - 1) == saf.SAF_ERR_WORKSPACE
    assert attn(lib, prefix=True, wsb=saf.paged_workspace_size(2, 4, 1, 2, 40) - 1) == saf.SAF_ERR_WORKSPACE
    assert attn(lib, ws=FAKE + 64) == bad
    assert attn(lib, B=1 << 15, T=1 << 15) == bad


def test_empty_calls(lib):
    for kw in (dict(B=0), dict(T=0)):
        assert append(lib, table=None, seq=None, q=None, k=None, v=None, **kw) == saf.SAF_OK
        assert attn(lib, table=None, seq=None, q=None, o=None, lse=None, ws=None, **kw) == saf.SAF_OK
    assert saf.paged_workspace_size(0, 4, 1, 2) == 0


def test_workspace_sizes(lib):
    assert lib.saf_paged_workspace_size(1, 4, 3, 1, 0) == ctypes.c_size_t(-1).value
    assert lib.saf_paged_workspace_size(1, 4, 4, 1, -1) == ctypes.c_size_t(-1).value
    small, large = saf.paged_workspace_size(1, 12, 1, 12), saf.paged_workspace_size(256, 32, 4, 8, 16384)
    assert 256 <= small <= large


def test_head_mask():
    assert saf.head_mask([0, 1, 0]) == b"\x00\x01\x00"
    assert saf.head_mask(torch.tensor([True, False])) == b"\x01\x00"
    assert saf.head_mask(b"\x01") == b"\x01"


def test_binding_refuses_host_tensors():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache"):
        saf.PagedKV(k, k)


def test_binding_refuses_a_prefix_without_pages():
    with pytest.raises(ValueError, match="prefix_table"):
        saf.paged_attn_prefix(None, None, None, 20, None, None)


def test_binding_refuses_a_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    cache = SimpleNamespace(device=torch.device("cuda", 0))
    other = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        saf.paged_attn(None, cache, None, None, stream=other)
    with pytest.raises(ValueError, match="stream"):
        saf.paged_attn_prefix(None, cache, torch.zeros(2), 20, None, None, stream=other)
    with pytest.raises(ValueError, match="stream"):
        saf.kv_append(None, None, None, cache, None, None, n_heads=1, stream=other)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: SimpleNamespace(device=torch.device("cuda", 0)))
    with pytest.raises(ValueError, match="stream"):
        saf.rope_table(4, stream=other)


def test_row_limit(lib):
    """Rows of a call are counted in 31 bits: a size below is wanted a workspace of, one past is refused by both calls."""
    bad, none = saf.SAF_ERR_INVALID_ARG, ctypes.c_size_t(-1).value
    for B, H, T in ((64, 4, 8192 * 8), (127, 4, 1 << 22)):
        assert attn(lib, B=B, H=H, T=T, wsb=0) == saf.SAF_ERR_WORKSPACE
        assert attn(lib, prefix=True, B=B, H=H, T=T, wsb=0) == saf.SAF_ERR_WORKSPACE
        rows = B * H * T
        assert rows * 66 * 4 < lib.saf_paged_workspace_size(B, H, 2, T, 40) < rows * 66 * 4 + (1 << 26)
    assert attn(lib, B=128, H=4, T=1 << 22, wsb=0) == bad
    assert attn(lib, prefix=True, B=128, H=4, T=1 << 22, wsb=0) == bad
    assert lib.saf_paged_workspace_size(128, 4, 2, 1 << 22, 0) == none
    assert lib.saf_paged_workspace_size(1, 256, 1, (1 << 25) - 1, 0) == none     # (256 times that is a multiple of 2^32, less 256)
    assert lib.saf_paged_workspace_size(1, 256, 1, 1 << 24, 40) == none


def test_device_status_waits_on_the_workspaces_device(monkeypatch):
    """Whatever device is current, as the serving calls run on their cache's."""
    entered, calls = [], []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *exc):
            entered.append(None)

    def status(ptr, nbytes, stream):
        calls.append((ptr, nbytes, stream, list(entered)))
        return saf.SAF_OK

    device = torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(saf, "_current_stream", lambda d: {device: 77}[d])
    monkeypatch.setattr(saf, "load", lambda: SimpleNamespace(saf_device_status=status))
    ws = SimpleNamespace(device=device, data_ptr=lambda: FAKE, numel=lambda: 512, element_size=lambda: 1)
    assert saf.device_status(ws) == saf.SAF_OK
    assert calls == [(FAKE, 512, 77, [device])] and entered == [device, None]
    with pytest.raises(ValueError, match="stream"):
        saf.device_status(ws, stream=SimpleNamespace(device=torch.device("cuda", 0)))
