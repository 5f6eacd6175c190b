"""The paged operators on many rows (prompt chunks, shared prefixes of large
batches), captured, with nothing to do and on several streams, against the fp64
loops of tests/paged_oracle.py.  Tolerances: see tests/test_paged_gpu.py; where a
row's maximum moves inside a block of keys, weights that were rounded already
are scaled and rounded once more, so that one more half step of bf16 is allowed.
"""
import math

import numpy as np
import pytest
import torch

from mixed_head_causal_b200 import saf
from tests import paged_oracle as O
from tests import parity as P
from tests.test_paged_gpu import S_TOL, U16, U32, Cache, check, np64, pattern, projections, run_attn

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("layout", ["heads", "slots", "pair"])
def test_chunks_ragged(page, layout):
    """q_lens from none to all of T, lengths at the edges of blocks, a group of each kind and a mixed one."""
    c = Cache([0, 40, 41, 127, 128, 129, 300, 20], 3, page, seed=page, layout=layout)
    run_attn(c, 6, 40, [0, 0, 1, 1, 0, 1], q_lens=[0, 40, 1, 33, 39, 40, 7, 40])


@pytest.mark.parametrize("H,Hkv,T,replaced", [(33, 1, 1, [32]), (5, 1, 7, [0, 4]), (64, 2, 2, range(32, 64)), (1, 1, 33, []),
                                              (1, 1, 200, [0]), (12, 4, 60, [1, 2, 3, 4, 5, 11])])
def test_chunks_head_layouts(H, Hkv, T, replaced):
    run_attn(Cache([T + 2, 260, T], Hkv, 32, seed=H), H, T, [h in replaced for h in range(H)])


@pytest.mark.parametrize("H,Hkv,T", [(256, 1, 1), (256, 256, 1), (256, 128, 20)])
@pytest.mark.parametrize("prefix", [0, 40])
def test_most_heads(H, Hkv, T, prefix):
    """256 heads: of one K/V head, each its own, two to one; every third replaced, and the last group."""
    mask = [int(h % 3 == 0 or h >= H - H // Hkv) for h in range(H)]
    run_attn(Cache([T + 3], Hkv, 16, seed=H, prefix=prefix), H, T, mask)


def test_chunk_bad_pages():
    c = Cache([200, 90, 140], 2, 16, seed=3)
    c.table[0, [0, 5, 12]] = [-1, c.kv.num_pages, -5]
    c.table[1, 2] = 2 ** 31 - 1
    c.table[2, :9] = -2 ** 31               # no key at all
    run_attn(c, 4, 40, [0, 1, 0, 0])


@pytest.mark.parametrize("T,prefix,lens", [(1, 0, [300, 9, 64]), (5, 0, [300, 9, 64]), (40, 0, [300, 41, 64]),
                                           (1, 139, [1 + 31 * i for i in range(40)]), (2, 139, [2 + i for i in range(40)])])
def test_unused_pattern_entries_are_not_read(T, prefix, lens):
    """NaN in the rows of ordinary heads and behind the longest position."""
    c = Cache(lens, 2, 16, seed=3, prefix=prefix)
    n = prefix + max(lens)
    a, r = pattern(4, n + 13, torch.Generator().manual_seed(5))
    for x in (a, r):
        x[:, n:] = float("nan")
        x[[0, 2]] = float("nan")
    run_attn(c, 4, T, [0, 1, 0, 1], a=a, r=r)


def test_thousands_of_sequences():
    g = np.random.default_rng(2)
    run_attn(Cache([int(n) for n in g.integers(0, 40, 4100)], 1, 16, seed=6, prefix=33), 1, 1, [0])


def test_chunk_infinite_patterns():
    c = Cache([150, 64, 300], 2, 16, seed=3)
    a, r = pattern(4, 300, torch.Generator().manual_seed(5))
    a[1, :140] = -float("inf")              # a whole block and more
    a[3] = -float("inf")                    # every row of head 3 empty
    r[2, 20:] = torch.finfo(torch.float32).min
    run_attn(c, 4, 40, [0, 1, 1, 1], a=a, r=r)


@pytest.mark.parametrize("prefix", [0, 256])
def test_maximum_moves_inside_a_block(prefix):
    """Scores that climb towards the first key by just under and just over the 2^8 that the maximum may lag."""
    c = Cache([256 - prefix // 2, 200], 1, 64, seed=3, prefix=prefix)
    n = prefix + 256
    T = 40
    bits = torch.tensor([0.0, 7.9, 8.2, 16.3, 16.6, 24.5, 33.0, 33.1])
    a = (torch.flip(bits, (0,)) * math.log(2)).repeat_interleave(32)
    a = torch.cat([a, torch.zeros(n - 256)]).repeat(2, 1).contiguous()
    a += 0.01 * torch.randn(2, n, generator=torch.Generator().manual_seed(1))
    r = torch.zeros(2, n)
    table, seq = c.gpu()
    q = torch.randn(2, 2, T, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    kw = dict(alpha=a.cuda(), rho=r.cuda(), mask=[1, 1], max_len=256)
    if prefix:
        o, lse = saf.paged_attn_prefix(q.cuda(), c.kv, torch.from_numpy(c.prefix_table).cuda(), prefix, table, seq, **kw)
    else:
        o, lse = saf.paged_attn(q.cuda(), c.kv, table, seq, **kw)
    ref = O.attend(np64(q), np64(c.k), np64(c.v), c.table, c.lens, None, np64(a), np64(r), [1, 1], 256, c.prefix_table, prefix)
    check(o, lse, ref, None, T, S_TOL + U16 / 2)
    assert (np.abs(np64(lse) - ref[1]) <= S_TOL + 2 * U32 * np.abs(ref[1])).all()


# ------------------------------------------------------------------ shared prefix
@pytest.mark.parametrize("T", [1, 2])
def test_prefix_far_positions(T):
    """Sequences whose lengths lie far apart (each row its own stretch of r), the last head's reaching r's end,
    and a pattern length that leaves no head but the first on a 16-byte boundary."""
    g = np.random.default_rng(1)
    lens = [int(n) for n in g.integers(T, 1500, 40)]
    lens[7], lens[8], lens[31] = 1501, T, 1500
    run_attn(Cache(lens, 2, 64, seed=4, prefix=523), 4, T, [0, 0, 1, 1], max_len=1501, n_pattern=2024 + 1)


def test_prefix_far_positions_end_of_r():
    """The same with a pattern of exactly the longest position's length."""
    lens = [1 + 37 * i for i in range(40)]
    run_attn(Cache(lens, 1, 64, seed=5, prefix=387), 2, 1, [0, 1], max_len=lens[-1])


@pytest.mark.parametrize("q_lens", [None, [40, 0, 13, 1, 40]])
def test_prefix_and_chunks(q_lens):
    c = Cache([40, 41, 170, 300, 45], 2, 32, seed=6, prefix=290)
    c.prefix_table[3] = -1
    c.table[2, 1] = c.kv.num_pages
    run_attn(c, 4, 40, [0, 1, 1, 1], q_lens=q_lens)


def test_prefix_only():
    """Nothing but the prefix: no columns in the page table, max_len 0."""
    c = Cache([0, 0, 0], 2, 32, seed=6, prefix=70, extra_cols=0)
    assert c.table.shape == (3, 0)
    run_attn(c, 4, 1, [0, 1, 0, 0], max_len=0)
    run_attn(c, 4, 20, [0, 1, 0, 0], max_len=0)


@pytest.mark.parametrize("T,B", [(1, 3), (40, 3), (1, 50)])
@pytest.mark.parametrize("prefix", [0, 200])
def test_no_new_tokens(T, B, prefix):
    """A call without a row leaves everything as it was, and the next ones on the stream have their turn."""
    H, mask = 4, [0, 1, 0, 0]
    c = Cache([T + 10 + i for i in range(B)], 2, 16, seed=6, prefix=prefix)
    ws = saf.new_paged_workspace(c.kv, B, H, T, prefix)
    table, seq = c.gpu()
    a, r = pattern(H, prefix + table.shape[1] * 16, torch.Generator().manual_seed(1))
    out, lse = torch.full((B, H, T, 64), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((B, H, T), 5.0, device="cuda")
    q = torch.randn(B, H, T, 64).bfloat16().cuda()
    kw = dict(alpha=a.cuda(), rho=r.cuda(), mask=mask, workspace=ws)
    pt = torch.from_numpy(c.prefix_table).cuda()

    def call(**more):
        if prefix:
            return saf.paged_attn_prefix(q, c.kv, pt, prefix, table, seq, **kw, **more)
        return saf.paged_attn(q, c.kv, table, seq, **kw, **more)

    want = [x.clone() for x in call()]
    none = ints([0] * B)
    for _ in range(8):
        call(q_lens=none, out=out, lse=lse)
        got = call()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (out == 5).all() and (lse == 5).all()
    assert saf.device_status(ws) == saf.SAF_OK


@pytest.mark.parametrize("prefix", [0, 20])
def test_rows_past_24_bits(prefix):
    """64 sequences of 8192 new tokens and 32 heads, all but the last of them before position 0."""
    B, H, Hkv, T, n = 64, 32, 8, 8192, 40
    mask = [int(h % 5 == 0) for h in range(H)]
    c = Cache([n] * B, Hkv, 16, seed=7, prefix=prefix)
    table, seq = c.gpu()
    a, r = pattern(H, prefix + n, torch.Generator().manual_seed(5))
    q = torch.zeros(B, H, T, 64, dtype=torch.bfloat16, device="cuda")
    some = prefix + n       # rows of a head that see a key
    q[:, :, -some:] = torch.randn(B, H, some, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    kw = dict(alpha=a.cuda(), rho=r.cuda(), mask=mask, max_len=n)
    ws = saf.new_paged_workspace(c.kv, B, H, T, prefix)
    if prefix:
        o, lse = saf.paged_attn_prefix(q, c.kv, torch.from_numpy(c.prefix_table).cuda(), prefix, table, seq, workspace=ws, **kw)
    else:
        o, lse = saf.paged_attn(q, c.kv, table, seq, workspace=ws, **kw)
    assert saf.device_status(ws) == saf.SAF_OK
    assert (o[:, :, :-some] == 0).all() and (lse[:, :, :-some] == -math.inf).all()
    for b in (0, 31, 63):
        ref = O.attend(np64(q[b:b + 1, :, -some:]), np64(c.k), np64(c.v), c.table[b:b + 1], [n], None, np64(a), np64(r), mask,
                       n, c.prefix_table, prefix)
        check(o[b:b + 1, :, -some:], lse[b:b + 1, :, -some:], ref, None, some)


@pytest.mark.parametrize("T", [1, 40])
def test_axis_limit(T):
    """The longest lengths that max_len allows bound the work: below 31 bits short sequences run, past them the call is refused."""
    page, H, max_len = 256, 2, 2 ** 31 - 2 ** 16
    c = Cache([300, 45], H, page, seed=2)
    q = torch.randn(40, H, T, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    table = torch.full((40, max_len // page), -1, dtype=torch.int32, device="cuda")
    table[:2, :c.table.shape[1]] = c.gpu()[0]
    seq = ints(c.lens + [0] * 38)
    B = 20 if T == 1 else 12     # 33.5 million tiles of 64 keys; blocks of 128 count twice
    o, lse = saf.paged_attn(q[:B].cuda(), c.kv, table[:B], seq[:B], max_len=max_len)
    ref = O.attend(np64(q[:B]), np64(c.k), np64(c.v), np.pad(c.table, ((0, B - 2), (0, 0))), c.lens + [0] * (B - 2), None, None, None,
                   [0] * H, 300)
    check(o, lse, ref, None, T)
    with pytest.raises(saf.SafError) as e:
        saf.paged_attn(q.cuda(), c.kv, table, seq, max_len=max_len)
    assert e.value.status == saf.SAF_ERR_UNSUPPORTED


BASE = 2 ** 30


@pytest.mark.parametrize("H,T,prefix,lens", [
    (1, 1, 0, [BASE + 300]), (2, 64, 0, [BASE + 300]),                      # one row, a chunk
    (1, 1, BASE, [300 + 37 * b for b in range(40)]), (2, 2, BASE, [300 + 37 * b for b in range(20)]),
    (1, 1, 256, [10 + b + BASE * (b % 2) for b in range(40)]),              # rows that far apart
])
def test_positions_past_30_bits(H, T, prefix, lens):
    """2^30 keys and more, the same pages over and over, under replaced heads whose pattern (two arrays of 4 GB a head)
    leaves weight near a row's own position alone: the fp64 formula over the last keys."""
    page, near, B = 256, 2000, len(lens)
    g = torch.Generator().manual_seed(B)
    kc, vc = (torch.randn(16, H, page, 64, generator=g).bfloat16() for _ in range(2))
    kv = saf.PagedKV(kc.cuda(), vc.cuda())
    n, cols = prefix + max(lens), -(-max(lens) // page)
    on_gpu = torch.Generator(device="cuda").manual_seed(1)
    pages = torch.randint(0, 16, (prefix // page,), generator=on_gpu, device="cuda", dtype=torch.int32)
    table = torch.randint(0, 16, (B, cols), generator=on_gpu, device="cuda", dtype=torch.int32)
    r = (torch.arange(n, device="cuda", dtype=torch.float32) * -0.05).repeat(H, 1)
    a = 0.5 * torch.randn(H, n, generator=on_gpu, device="cuda")
    q = torch.zeros(B, H, T, 64, dtype=torch.bfloat16, device="cuda")
    kw = dict(alpha=a, rho=r, mask=[1] * H, max_len=max(lens))
    if prefix:
        o, lse = saf.paged_attn_prefix(q, kv, pages, prefix, table, ints(lens), **kw)
    else:
        o, lse = saf.paged_attn(q, kv, table, ints(lens), **kw)
    v64 = np64(vc)
    for b in range(B):
        for t in range(T):
            i = prefix + lens[b] - T + t
            j = torch.arange(max(0, i - near), i + 1, device="cuda")
            at = torch.where(j < prefix, pages[torch.clamp(j // page, max=prefix // page - 1)] if prefix else 0,
                             table[b][torch.clamp(j - prefix, min=0) // page]).cpu().numpy()
            slot = (torch.where(j < prefix, j, j - prefix) % page).cpu().numpy()
            for h in range(H):
                v = v64[at, h, slot]
                s = np64(a[h, j]) - 0.05 * np64(i - j)
                w = np.exp(s - s.max())
                want, total = w @ v / w.sum(), s.max() + np.log(w.sum())
                bound = U16 * np.abs(want) + (U16 + 2 * S_TOL) * (w @ np.abs(v) / w.sum())
                assert (np.abs(np64(o[b, h, t]) - want) <= bound).all(), (b, h, t)
                assert abs(float(lse[b, h, t]) - total) <= S_TOL + 2 * U32 * abs(total)


# ------------------------------------------------------------------ together
def test_prefill_by_chunks_matches_the_layer():
    """A prompt appended and attended chunk by chunk, ragged last chunks included: the layer's own rows."""
    B, H, Hkv, page, C = 2, 4, 2, 32, 48
    lens, T = [150, 97], 150
    mask = [0, 1, 0, 0]
    g = torch.Generator().manual_seed(3)
    q, k, v = projections(B, H, Hkv, T, g, "tokens")
    a, r = (x.cuda() for x in pattern(H, T, g))
    rope = saf.rope_table(T)
    cols = -(-T // page)
    kv = saf.PagedKV(*(torch.full((B * cols, Hkv, page, 64), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    other = saf.PagedKV(kv.k_cache.clone(), kv.v_cache.clone())
    table = torch.randperm(B * cols, generator=g).to(torch.int32).view(B, cols).cuda()
    k_rot = torch.zeros(B, Hkv, T, 64, dtype=torch.bfloat16, device="cuda")
    q_rot, _ = saf.kv_append(q, k, v, other, table, ints([T] * B), mask=mask, rope=rope, max_len=T, k_out=k_rot)
    o_all, lse_all = saf.mixed_attn_fwd(q_rot, k_rot, v.contiguous(), a, r, mask)
    ws = saf.new_paged_workspace(kv, B, H, C)
    for t0 in range(0, T, C):
        n = [max(0, min(C, x - t0)) for x in lens]
        seq, ql = ints([min(x, t0 + C) for x in lens]), ints(n)
        t1 = min(t0 + C, T)
        qc = torch.zeros(B, H, C, 64, dtype=torch.bfloat16, device="cuda")
        kc, vc = (torch.zeros(B, Hkv, C, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for dst, src in ((qc, q), (kc, k), (vc, v)):
            dst[:, :, :t1 - t0] = src[:, :, t0:t1]
        qr, _ = saf.kv_append(qc, kc, vc, kv, table, seq, mask=mask, q_lens=ql, rope=rope, max_len=T)
        o, lse = saf.paged_attn(qr, kv, table, seq, alpha=a, rho=r, mask=mask, q_lens=ql, max_len=T, workspace=ws)
        for b in range(B):
            at = slice(t0, t0 + n[b])
            assert (o[b, :, :n[b]].float() - o_all[b, :, at].float()).abs().max() <= P.TOL_MAX if n[b] else True
            assert (lse[b, :, :n[b]] - lse_all[b, :, at]).abs().max() <= P.TOL_LSE if n[b] else True
            assert (o[b, :, n[b]:] == 0).all()
    assert saf.device_status(ws) == saf.SAF_OK


@pytest.mark.parametrize("T", [1, 40])
def test_captured_prefix_calls_share_a_workspace(T):
    """Two captured calls of different batches behind prefixes of their own; replays follow lengths and queries."""
    H, mask = 4, [0, 1, 0, 0]
    caches = [Cache([300, 40, 129], 2, 16, seed=1, prefix=333), Cache([64 + 3 * i for i in range(20)], 2, 16, seed=2, prefix=100)]
    a, r = pattern(H, 700, torch.Generator().manual_seed(2))
    ag, rg = a.cuda(), r.cuda()
    ws = saf.new_paged_workspace(caches[0].kv, 20, H, T, 333)
    runs = []
    for c in caches:
        B = len(c.lens)
        table, seq = c.gpu()
        pt = torch.from_numpy(c.prefix_table).cuda()
        q = torch.zeros(B, H, T, 64, dtype=torch.bfloat16, device="cuda")
        out, lse, ql = torch.zeros_like(q), torch.zeros(B, H, T, device="cuda"), ints([T] * B)

        def step(c=c, q=q, out=out, lse=lse, table=table, seq=seq, pt=pt, ql=ql):
            saf.paged_attn_prefix(q, c.kv, pt, c.prefix, table, seq, alpha=ag, rho=rg, mask=mask, q_lens=ql, out=out,
                                  lse=lse, workspace=ws)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((c, graph, q, out, lse, seq, ql, step))     # (step holds the tables that the graph reads)
    for k in range(3):
        for c, graph, q, out, lse, seq, ql, _ in runs:
            lens = [max(0, n - 37 * k) for n in c.lens]
            q_lens = [T if k != 1 else 0] * len(lens)
            seq.copy_(ints(lens))
            ql.copy_(ints(q_lens))
            new = torch.randn(q.shape, generator=torch.Generator().manual_seed(k)).bfloat16()
            q.copy_(new)
        for c, graph, q, out, lse, seq, ql, _ in runs:     # back to back
            graph.replay()
        torch.cuda.synchronize()
        for c, graph, q, out, lse, seq, ql, _ in runs:
            ref = O.attend(np64(q), np64(c.k), np64(c.v), c.table, seq.tolist(), ql.tolist(), np64(a), np64(r), mask, 300,
                           c.prefix_table, c.prefix)
            check(out, lse, ref, ql.tolist(), T)
    assert saf.device_status(ws) == saf.SAF_OK


def test_calls_at_once_on_two_streams():
    """Chunks and single tokens on two streams at the same time, a workspace each: the results of either alone."""
    big, small = Cache([700, 640, 900], 2, 64, seed=1), Cache([300, 40, 129], 2, 16, seed=2, prefix=400)
    qb, qs = torch.randn(3, 4, 64, 64).bfloat16().cuda(), torch.randn(3, 4, 1, 64).bfloat16().cuda()
    (tb, sb), (ts, ss) = big.gpu(), small.gpu()
    pt = torch.from_numpy(small.prefix_table).cuda()
    want_b = saf.paged_attn(qb, big.kv, tb, sb, max_len=900)
    want_s = saf.paged_attn_prefix(qs, small.kv, pt, 400, ts, ss, max_len=300)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((saf.paged_attn(qb, big.kv, tb, sb, max_len=900, stream=s1), want_b))
        got.append((saf.paged_attn_prefix(qs, small.kv, pt, 400, ts, ss, max_len=300, stream=s2), want_s))
    torch.cuda.synchronize()
    for (o, lse), want in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_sequences_share_pages():
    """The same pages in several rows of the table, and one page twice in a row: read as they stand."""
    c = Cache([130, 130, 64], 2, 32, seed=4)
    c.table[1] = c.table[0]
    c.table[2, 1] = c.table[2, 0]
    run_attn(c, 4, 1, [0, 1, 0, 0])
    run_attn(c, 4, 40, [0, 1, 0, 0])


def test_views_of_the_callers_tensors():
    """Tables, lengths and outputs that are slices at odd offsets of larger tensors."""
    c = Cache([130, 33, 64], 2, 32, seed=4)
    table, seq = c.gpu()
    cols = table.shape[1]
    flat = torch.full((3 * cols + 1,), -9, dtype=torch.int32, device="cuda")
    flat[1:] = table.flatten()
    nums = torch.cat([ints([7]), seq, ints([1, 1, 1])])
    q = torch.randn(3, 4, 1, 64).bfloat16()
    o, lse = saf.paged_attn(q.cuda(), c.kv, flat[1:].view(3, cols), nums[1:4], q_lens=nums[4:], max_len=130)
    ref = O.attend(np64(q), np64(c.k), np64(c.v), c.table, c.lens, None, None, None, [0] * 4, 130)
    check(o, lse, ref, None, 1)


def test_in_place_rotation():
    """Contiguous queries may be rotated where they stand."""
    c = Cache([5, 33], 2, 16, seed=4)
    table, seq = c.gpu()
    rope = saf.rope_table(40)
    for inter in (False, True):
        q = torch.randn(2, 4, 3, 64).bfloat16().cuda()
        k, v = (torch.randn(2, 2, 3, 64).bfloat16().cuda() for _ in range(2))
        want, _ = saf.kv_append(q, k, v, c.kv, table, seq, rope=rope, interleaved=inter, max_len=33)
        got, _ = saf.kv_append(q, k, v, c.kv, table, seq, rope=rope, interleaved=inter, max_len=33, q_out=q)
        assert got is q and torch.equal(want, q)


def test_chunks_repeatable():
    c = Cache([900, 400, 129, 333], 2, 16, seed=1)
    q = torch.randn(4, 8, 60, 64).bfloat16().cuda()
    table, seq = c.gpu()
    a, r = (x.cuda() for x in pattern(8, 900, torch.Generator().manual_seed(1)))
    kw = dict(alpha=a, rho=r, mask=[0, 1] * 4, max_len=900)
    first = saf.paged_attn(q, c.kv, table, seq, **kw)
    for _ in range(10):
        again = saf.paged_attn(q, c.kv, table, seq, **kw)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
