"""The serving operators (paged cache append, paged attention, shared-prefix
attention) on the GPU against plain fp64 loops (tests/paged_oracle.py).

Tolerances, from the arithmetic (u = half a step: 2^-8 in bf16, 2^-24 in fp32):
  * rotated values: one bf16 rounding of the result, 2^-8 |y|, and three fp32
    operations on the two products, 3 u32 (|x0 c| + |x1 s|) <= 3 u32 (|x0| + |x1|);
    what is only copied is equal;
  * lse: a score is a sum of 64 exact products in fp32, off by at most
    64 u32 sum|q_c k_c| / 8 (replaced: one rounding, u32 |s|), its logarithm of
    a sum of n exponentials by n u32 + 2^-22 more; S_TOL below bounds it for
    the sizes here: sum|q k| / 8 < 8 gives 3.1e-5, n < 4096 gives 2.5e-4 at the very
    worst and (the signs of n roundings being independent) sqrt(n) u32 < 4e-6 in
    earnest; 1e-4 is used, and 2 u32 |lse| for the final operations;
  * o: each weight is rounded to bf16 at most once (u16 relative) and carries
    the score's error twice (its own and the row sum's): (2^-8 + 2 S_TOL)
    sum P|v|, and the result's own rounding 2^-8 |o|.
"""
import numpy as np
import pytest
import torch

from mixed_head_causal_b200 import inputs as I
from mixed_head_causal_b200 import saf
from tests import paged_oracle as O
from tests import parity as P

pytestmark = pytest.mark.gpu

U16, U32, S_TOL = 2.0 ** -8, 2.0 ** -24, 1e-4
STALE = float("nan")


def np64(t):
    return t.detach().cpu().double().numpy()


class Cache:
    """A random paged cache: lens tokens per sequence behind a shared prefix,
    pages in random order, NaN in every slot that holds no token."""

    def __init__(self, lens, Hkv, page, seed=0, prefix=0, spare=3, layout="heads", extra_cols=1):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        pp = -(-prefix // page)
        total = sum(need) + pp + spare
        order = torch.randperm(total, generator=g).tolist()
        cols = max(need + [0]) + extra_cols
        table = np.full((len(lens), cols), -7, dtype=np.int32)
        live = np.zeros((total, page), dtype=bool)

        def fill(n):
            row = [order.pop() for _ in range(-(-n // page))]
            for j in range(n):
                live[row[j // page], j % page] = True
            return row

        self.prefix_table = np.array(fill(prefix), dtype=np.int32)
        for b, n in enumerate(lens):
            row = fill(n)
            table[b, :len(row)] = row
        k, v = (torch.randn(total, Hkv, page, 64, generator=g).bfloat16() for _ in range(2))
        dead = torch.from_numpy(~live)[:, None, :, None]
        self.k, self.v = self.lay_out(k.masked_fill(dead, STALE), layout), self.lay_out(v.masked_fill(dead, STALE), layout)
        self.kv = saf.PagedKV(self.k, self.v)
        self.table, self.lens, self.prefix, self.g = table, list(lens), prefix, g
        self.page = page

    @staticmethod
    def lay_out(x, layout):
        if layout == "heads":       # [pages, heads, slots, 64]
            return x.cuda()
        if layout == "slots":       # stored [pages, slots, heads, 64]
            return x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        big = torch.full((x.shape[0], 2, x.shape[1], x.shape[2], 64), STALE, dtype=torch.bfloat16, device="cuda")
        big[:, 1] = x.cuda()        # one half of a tensor that holds K and V pages side by side
        return big[:, 1]

    def gpu(self):
        return (torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda"))


def pattern(H, n, g):
    a = torch.randn(H, n, generator=g) * 0.5
    r = -0.05 * torch.arange(n).float() + 0.3 * torch.randn(H, n, generator=g)
    a[:, 0] += 4
    r[:, 0] += 2
    return a, r


def check(o, lse, ref, q_lens, T, s_tol=S_TOL):
    o_ref, lse_ref, w = ref
    o, lse = np64(o), np64(lse)
    for b in range(o.shape[0]):
        n = O.new_tokens(q_lens, b, T)
        if n == 0:
            continue
        got, want, wt = o[b, :, :n], o_ref[b, :, :n], w[b, :, :n]
        assert np.isfinite(got).all(), f"sequence {b}: non-finite output"
        over = np.abs(got - want) - (U16 * np.abs(want) + (U16 + 2 * s_tol) * wt)
        assert over.max() <= 0, f"sequence {b}: o off by {np.abs(got - want).max():.3e}"
        gl, wl = lse[b, :, :n], lse_ref[b, :, :n]
        empty = np.isneginf(wl)
        assert (np.isneginf(gl) == empty).all(), f"sequence {b}: empty rows"
        assert (got[empty] == 0).all()
        gl, wl = gl[~empty], wl[~empty]
        assert (np.abs(gl - wl) <= s_tol + 2 * U32 * np.abs(wl)).all(), f"sequence {b}: lse off by {np.abs(gl - wl).max():.3e}"


def run_attn(c, H, T, mask, q_lens=None, seed=1, max_len=None, workspace=None, n_pattern=None, a=None, r=None, q=None):
    g = torch.Generator().manual_seed(seed)
    B = len(c.lens)
    table, seq = c.gpu()
    max_len = max_len if max_len is not None else max(max(c.lens), 1)
    q = torch.randn(B, H, T, 64, generator=g).bfloat16() if q is None else q
    if a is None:
        a, r = pattern(H, n_pattern or c.prefix + max_len, g)
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device="cuda")
    out = torch.full((B, H, T, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, T), 5.0, device="cuda")
    qg = q.clone()
    qg[:, [h for h in range(H) if mask[h]]] = STALE     # a replaced head's q is not read
    kw = dict(alpha=a.cuda(), rho=r.cuda(), mask=mask, q_lens=ql, max_len=max_len, out=out, lse=lse, workspace=workspace)
    if c.prefix:
        saf.paged_attn_prefix(qg.cuda(), c.kv, torch.from_numpy(c.prefix_table).cuda(), c.prefix, table, seq, **kw)
    else:
        saf.paged_attn(qg.cuda(), c.kv, table, seq, **kw)
    torch.cuda.synchronize()
    ref = O.attend(np64(q), np64(c.k), np64(c.v), c.table, c.lens, q_lens, np64(a), np64(r), mask, max_len,
                   c.prefix_table, c.prefix)
    check(out, lse, ref, q_lens, T)
    for b in range(B):      # rows behind a sequence's tokens are left as they were
        n = O.new_tokens(q_lens, b, T)
        assert (out[b, :, n:] == 5).all() and (lse[b, :, n:] == 5).all()
    return out, lse


# ------------------------------------------------------------------ append
def projections(B, H, Hkv, T, g, layout):
    if layout == "tokens":      # slices of one projection's output, token-major
        qkv = torch.randn(B, T, H + 2 * Hkv, 64, generator=g).bfloat16().cuda().transpose(1, 2)
        return qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    return tuple(torch.randn(B, h, T, 64, generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv))


@pytest.mark.parametrize("B,H,Hkv,T,page,lens,q_lens,replaced,rot,inter,offset,layout,cache", [
    (1, 1, 1, 1, 16, [1], None, [], 64, False, 0, "heads", "heads"),
    (3, 4, 4, 1, 64, [1, 64, 65], None, [2], 64, False, 0, "tokens", "heads"),
    (2, 6, 2, 5, 16, [5, 37], None, [0, 1, 2], 32, False, 0, "tokens", "slots"),
    (3, 4, 2, 33, 32, [33, 90, 40], [33, 0, 7], [1], 64, True, 11, "heads", "heads"),
    (2, 3, 3, 70, 128, [70, 200], [70, 69], [0, 1, 2], 48, False, 0, "heads", "pair"),
    (2, 4, 1, 17, 256, [17, 300], [16, 17], [], 16, True, 5, "tokens", "pair"),
    (2, 2, 2, 9, 16, [9, 20], None, [1], 0, False, 0, "heads", "slots"),
])
def test_append(B, H, Hkv, T, page, lens, q_lens, replaced, rot, inter, offset, layout, cache):
    g = torch.Generator().manual_seed(B * 100 + T)
    c = Cache(lens, Hkv, page, seed=T, layout=cache)
    mask = [h in replaced for h in range(H)]
    q, k, v = projections(B, H, Hkv, T, g, layout)
    max_len = max(lens)
    rope = saf.rope_table(offset + max_len, rot) if rot else None
    q_out, k_out = (torch.full((B, h, T, 64), 5.0, dtype=torch.bfloat16, device="cuda") for h in (H, Hkv))
    before = [np64(q_out), np64(k_out), np64(c.k), np64(c.v)]
    table, seq = c.gpu()
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device="cuda")
    saf.kv_append(q, k, v, c.kv, table, seq, mask=mask, q_lens=ql, rope=rope, interleaved=inter, max_len=max_len,
                  pos_offset=offset, q_out=q_out, k_out=k_out)
    got = [np64(x) for x in (q_out, k_out, c.k, c.v)]
    ref = [x.copy() for x in before]
    O.append(np64(q), np64(k), np64(v), ref[2], ref[3], c.table, lens, q_lens, None if rope is None else np64(rope),
             inter, mask, max_len, offset, ref[0], ref[1])
    np.testing.assert_array_equal(got[3], ref[3])       # V is copied
    big = max(float(np.abs(np64(x)).max()) for x in (q, k))
    for x, y, old in zip(got[:3], ref[:3], before[:3]):
        same = (y == old) | (np.isnan(y) & np.isnan(old))
        np.testing.assert_array_equal(x[same], y[same])     # what no token reaches is untouched
        tol = U16 * np.abs(y) + 3 * U32 * 2 * big if rot else np.zeros_like(y)
        assert (np.abs(x - y) <= tol)[~same].all()


def test_rope_table_far_positions():
    got = np64(saf.rope_table(200_001, 64, 500_000.0))
    for p in (0, 1, 4095, 131_071, 200_000):
        w = 500_000.0 ** (-np.arange(32) / 32.0)
        # the fp64 angle is off by p w 2^-52 and a little more, the result by half an fp32 step
        np.testing.assert_allclose(got[p], np.concatenate([np.cos(p * w), np.sin(p * w)]), rtol=0, atol=U32 + 1e-9)


def test_append_skips_bad_pages_and_positions():
    c = Cache([40, 40], 2, 16, seed=3)
    c.table[0, 1] = -1                      # positions 16..31 of sequence 0 have no page
    c.table[1, 2] = c.kv.num_pages          # positions 32..39 of sequence 1 neither
    g = torch.Generator().manual_seed(0)
    q, k, v = projections(2, 2, 2, 40, g, "heads")
    before = [np64(c.k), np64(c.v)]
    table, _ = c.gpu()
    seq = torch.tensor([40, 43], dtype=torch.int32, device="cuda")  # 43: three tokens past max_len
    q_out, _ = saf.kv_append(q, k, v, c.kv, table, seq, max_len=40)
    ref = [x.copy() for x in before]
    q_ref = np.zeros(q.shape)
    O.append(np64(q), np64(k), np64(v), *ref, c.table, [40, 43], None, None, False, [0, 0], 40, 0, q_ref, None)
    np.testing.assert_array_equal(np64(c.k), ref[0])
    np.testing.assert_array_equal(np64(c.v), ref[1])
    np.testing.assert_array_equal(np64(q_out), q_ref)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,Hkv,replaced", [(3, 3, [1]), (4, 2, [0, 1]), (6, 1, [5]), (2, 2, [])],
                         ids=["h3_r1", "gqa2_group_replaced", "mqa6_r1", "h2_plain"])
def test_decode_lengths(page, H, Hkv, replaced):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 700]
    run_attn(Cache(lens, Hkv, page, seed=page), H, 1, [h in replaced for h in range(H)])


@pytest.mark.parametrize("H,Hkv,T,replaced", [
    (4, 4, 2, [1]), (12, 3, 5, [0, 1, 2, 3, 7]), (8, 1, 8, [3]), (8, 2, 16, [0]), (2, 2, 67, [1]), (6, 2, 130, [0, 1, 2, 4]),
    (3, 3, 300, [2])])
def test_several_new_tokens(H, Hkv, T, replaced):
    lens = [T, T + 1, T + 63, 2 * T + 40, 500]
    lens = [max(n, T) for n in lens]
    run_attn(Cache(lens, Hkv, 32, seed=T), H, T, [h in replaced for h in range(H)])


def test_ragged_new_tokens():
    lens = [9, 0, 30, 129, 4]
    run_attn(Cache(lens, 2, 16, seed=8), 4, 9, [0, 1, 0, 0], q_lens=[9, 0, 1, 5, 4])
    # more new tokens than the cache holds: the rows before position 0 are empty
    run_attn(Cache([3, 0, 70], 2, 16, seed=9), 4, 9, [0, 1, 0, 0], q_lens=[9, 2, 9])
    # q_lens outside [0, T] are clamped, seq_lens past max_len too
    run_attn(Cache([30, 50], 2, 16, seed=9), 4, 3, [0, 1, 0, 0], q_lens=[7, -2], max_len=41)


def test_long_context_few_rows():
    """One long sequence among short ones: the key axis is split and joined."""
    run_attn(Cache([3500, 3, 0, 640], 2, 64, seed=4), 2, 1, [0, 1])
    run_attn(Cache([2900], 1, 16, seed=5), 1, 1, [0])


def test_large_batch():
    g = np.random.default_rng(0)
    run_attn(Cache([int(n) for n in g.integers(0, 90, 333)], 2, 32, seed=6), 4, 1, [0, 0, 1, 0])


@pytest.mark.parametrize("layout", ["slots", "pair"])
def test_cache_layouts(layout):
    run_attn(Cache([100, 33, 257], 3, 32, seed=2, layout=layout), 6, 2, [0, 0, 1, 0, 0, 0])


def test_bad_pages_are_left_out():
    c = Cache([200, 90, 40], 2, 16, seed=3)
    c.table[0, [0, 5]] = [-1, c.kv.num_pages]
    c.table[1, 2] = 2 ** 31 - 1
    c.table[2, :3] = -2 ** 31               # no key at all
    run_attn(c, 4, 3, [0, 1, 0, 0])


def test_rows_of_minus_infinity_and_lowest():
    c = Cache([150, 64, 10], 2, 16, seed=3)
    a, r = pattern(2, 150, torch.Generator().manual_seed(5))
    a[1, :20] = -float("inf")
    a[1, 20:40] = torch.finfo(torch.float32).min
    run_attn(c, 2, 1, [0, 1], a=a, r=r)
    a[1] = -float("inf")                    # every row of head 1 empty
    run_attn(c, 2, 1, [0, 1], a=a, r=r)
    a[1] = torch.finfo(torch.float32).min / 2   # uniform a, far below anything: the softmax does not mind
    run_attn(c, 2, 1, [0, 1], a=a, r=torch.zeros_like(r))


def test_peaked_scores():
    """Scores in the hundreds: one key takes all the weight, the rest underflow."""
    c = Cache([300, 129], 2, 16, seed=3)
    q = 30 * torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    table, seq = c.gpu()
    o, lse = saf.paged_attn(q.cuda(), c.kv, table, seq, max_len=300)
    ref = O.attend(np64(q), np64(c.k), np64(c.v), c.table, c.lens, None, None, None, [0] * 4, 300)
    # the score's bound of the heading, with this case's largest sum|q k| / 8
    k = np.abs(np.nan_to_num(np64(c.k))).reshape(-1, 64)
    s_tol = 64 * U32 * (np.abs(np64(q)).reshape(-1, 64) @ k.T).max() / 8
    check(o, lse, ref, None, 1, s_tol + S_TOL)


@pytest.mark.parametrize("B,H,Hkv,T,prefix,lens,replaced,page", [
    (1, 2, 2, 1, 100, [1], [1], 16),
    (3, 4, 4, 1, 64, [0, 5, 130], [0], 64),             # a sequence with nothing of its own
    (5, 4, 2, 1, 777, [3, 90, 1, 64, 200], [2, 3], 32),
    (9, 8, 2, 3, 300, [3, 10, 5, 4, 3, 77, 30, 3, 20], [0, 5], 16),
    (40, 4, 1, 1, 500, list(range(1, 41)), [1], 128),
    (70, 3, 3, 2, 1000, [2 + i % 30 for i in range(70)], [2], 64),
    (33, 8, 1, 4, 129, [4 + i for i in range(33)], [], 16),
])
def test_shared_prefix(B, H, Hkv, T, prefix, lens, replaced, page):
    run_attn(Cache(lens, Hkv, page, seed=B, prefix=prefix), H, T, [h in replaced for h in range(H)])


def test_shared_prefix_ragged_and_bad_pages():
    c = Cache([9, 3, 40, 1], 2, 16, seed=5, prefix=90)
    c.prefix_table[2] = -1
    run_attn(c, 4, 4, [0, 1, 0, 0], q_lens=[4, 0, 2, 4])


def test_prefix_equals_the_same_keys_unshared():
    """Copies of the prefix in every sequence's own pages give the same rows."""
    shared = Cache([7, 50, 33], 2, 16, seed=5, prefix=160)
    own = Cache([167, 210, 193], 2, 16, seed=6)
    for b, n in enumerate(shared.lens):
        for j in range(160 + n):
            src = (shared.prefix_table[j // 16], j % 16) if j < 160 else (shared.table[b, (j - 160) // 16], (j - 160) % 16)
            for x, y in ((own.k, shared.k), (own.v, shared.v)):
                x[int(own.table[b, j // 16]), :, j % 16] = y[int(src[0]), :, int(src[1])]
    a, r = pattern(4, 260, torch.Generator().manual_seed(2))
    q = torch.randn(3, 4, 1, 64).bfloat16()
    o1, l1 = run_attn(shared, 4, 1, [0, 1, 0, 0], a=a, r=r, q=q)
    o2, l2 = run_attn(own, 4, 1, [0, 1, 0, 0], a=a, r=r, q=q)
    assert (l1 - l2).abs().max() <= 2 * S_TOL


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("Hkv", [4, 2])
def test_prefill_then_decode_matches_the_layer(Hkv):
    """Prefill with the layer, append, then decode token by token: the rows are
    the layer's own rows over the whole sequence."""
    B, H, T0, steps, page = 2, 4, 150, 5, 32
    mask = [0, 1, 0, 0]
    g = torch.Generator().manual_seed(3)
    T = T0 + steps
    q, k, v = projections(B, H, Hkv, T, g, "heads")
    a, r = (x.cuda() for x in pattern(H, T, g))
    rope = saf.rope_table(T)
    cols = -(-T // page)
    kc, vc = (torch.full((B * cols, Hkv, page, 64), STALE, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv = saf.PagedKV(kc, vc)
    table = torch.randperm(B * cols, generator=g).to(torch.int32).view(B, cols).cuda()
    # the whole sequence at once, rotated through another cache
    other = saf.PagedKV(kc.clone(), vc.clone())
    full = torch.full((B,), T, dtype=torch.int32, device="cuda")
    k_rot = torch.zeros_like(k)
    q_rot, _ = saf.kv_append(q, k, v, other, table, full, mask=mask, rope=rope, max_len=T, k_out=k_rot)
    o_all, lse_all = saf.mixed_attn_fwd(q_rot, k_rot, v, a, r, mask)
    # prompt, then single tokens
    seq = torch.full((B,), T0, dtype=torch.int32, device="cuda")
    q0, k0, v0 = (x[:, :, :T0] for x in (q, k, v))
    k0_rot = torch.zeros(B, Hkv, T0, 64, dtype=torch.bfloat16, device="cuda")
    q0_rot, _ = saf.kv_append(q0, k0, v0, kv, table, seq, mask=mask, rope=rope, max_len=T, k_out=k0_rot)
    assert torch.equal(q0_rot, q_rot[:, :, :T0])
    ar, rr = a[:, :T0].contiguous(), r[:, :T0].contiguous()
    o0, _ = saf.mixed_attn_fwd(q0_rot, k0_rot, v0.contiguous(), ar, rr, mask)
    assert (o0.float() - o_all[:, :, :T0].float()).abs().max() <= P.TOL_MAX
    ws = saf.new_paged_workspace(kv, B, H)
    for t in range(T0, T):
        seq += 1
        q1, _ = saf.kv_append(q[:, :, t:t + 1], k[:, :, t:t + 1], v[:, :, t:t + 1], kv, table, seq, mask=mask, rope=rope,
                              max_len=T)
        o1, lse1 = saf.paged_attn(q1, kv, table, seq, alpha=a, rho=r, mask=mask, max_len=T, workspace=ws)
        assert (o1.float() - o_all[:, :, t:t + 1].float()).abs().max() <= P.TOL_MAX
        assert (lse1 - lse_all[:, :, t:t + 1]).abs().max() <= P.TOL_LSE
    for x, y in ((kc, other.k_cache), (vc, other.v_cache)):
        assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(), y.nan_to_num())


def test_graphs_share_a_workspace_and_follow_the_lengths():
    """Two captured steps (different batches) share a workspace; replays see new lengths, queries and tables."""
    caches = [Cache([300, 40, 129], 2, 16, seed=1, extra_cols=4), Cache([64, 500], 2, 16, seed=2, extra_cols=4)]
    H, mask = 4, [0, 1, 0, 0]
    a, r = pattern(H, 600, torch.Generator().manual_seed(2))
    ag, rg = a.cuda(), r.cuda()
    ws = saf.new_paged_workspace(caches[0].kv, 3, H)
    runs = []
    for c in caches:
        B = len(c.lens)
        table, seq = c.gpu()
        q = torch.zeros(B, H, 1, 64, dtype=torch.bfloat16, device="cuda")
        out, lse = torch.zeros_like(q), torch.zeros(B, H, 1, device="cuda")

        def step(c=c, q=q, out=out, lse=lse, table=table, seq=seq):
            saf.paged_attn(q, c.kv, table, seq, alpha=ag, rho=rg, mask=mask, max_len=table.shape[1] * 16,
                           out=out, lse=lse, workspace=ws)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((c, graph, q, out, lse, table, seq))
    for k in range(3):
        for c, graph, q, out, lse, table, seq in runs:
            lens = [max(0, n - 37 * k) for n in c.lens]
            seq.copy_(torch.tensor(lens, dtype=torch.int32))
            new = torch.randn(q.shape, generator=torch.Generator().manual_seed(k)).bfloat16()
            q.copy_(new)
            graph.replay()
            ref = O.attend(np64(new), np64(c.k), np64(c.v), c.table, lens, None, np64(a), np64(r), mask, 600)
            check(out, lse, ref, None, 1)
    assert saf.device_status(ws) == saf.SAF_OK


def test_another_stream():
    c = Cache([300, 40, 129], 2, 16, seed=1)
    q = torch.randn(3, 4, 1, 64).bfloat16().cuda()
    table, seq = c.gpu()
    base = saf.paged_attn(q, c.kv, table, seq, max_len=300)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(20):     # every call allocates its outputs and workspace on the stream it runs on
        got.append(saf.paged_attn(q, c.kv, table, seq, max_len=300, stream=s))
    s.synchronize()
    for o, lse in got:
        assert torch.equal(o, base[0]) and torch.equal(lse, base[1])


def test_repeatable():
    c = Cache([900, 40, 129, 333], 2, 16, seed=1, prefix=400)
    q = torch.randn(4, 4, 2, 64).bfloat16().cuda()
    table, seq = c.gpu()
    pt = torch.from_numpy(c.prefix_table).cuda()
    first = saf.paged_attn_prefix(q, c.kv, pt, 400, table, seq, max_len=900)
    for _ in range(10):
        again = saf.paged_attn_prefix(q, c.kv, pt, 400, table, seq, max_len=900)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31 (a cache of over 4 GB)."""
    page, Hkv = 64, 4
    n = (2 ** 31) // (page * Hkv * 64) + 40
    k, v = (torch.empty(n, Hkv, page, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv = saf.PagedKV(k, v)
    c = Cache([130, 64], Hkv, page, seed=3, spare=0)
    far = n - c.kv.num_pages
    k[far:], v[far:] = c.k, c.v
    q = torch.randn(2, 4, 1, 64).bfloat16()
    _, seq = c.gpu()
    table = torch.from_numpy(np.where(c.table >= 0, c.table + far, -1).astype(np.int32)).cuda()
    o, lse = saf.paged_attn(q.cuda(), kv, table, seq, max_len=130)
    ref = O.attend(np64(q), np64(c.k), np64(c.v), c.table, c.lens, None, None, None, [0] * 4, 130)
    check(o, lse, ref, None, 1)
    new = torch.randn(2, Hkv, 1, 64).bfloat16().cuda()
    saf.kv_append(None, new, new, kv, table, seq, max_len=130)
    assert torch.equal(k[int(table[0, 2]), :, 1], new[0, :, 0]) and torch.equal(v[int(table[1, 0]), :, 63], new[1, :, 0])
