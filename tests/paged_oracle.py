"""The serving operators in plain fp64 loops on the CPU, for the tests: the
cache is read slot by slot through its page table, every row on its own."""
import math

import numpy as np

HEAD_DIM = 64


def new_tokens(q_lens, b, T):
    return T if q_lens is None else min(max(int(q_lens[b]), 0), T)


def append(q, k, v, k_cache, v_cache, page_table, seq_lens, q_lens, rope, interleaved, mask, max_len, pos_offset,
           q_out, k_out):
    """All arrays fp64 (tables int); k_cache, v_cache [pages, H_kv, page, 64], q_out, k_out are updated."""
    B, Hkv, T, _ = k.shape
    H = q.shape[1]
    group, page_size, rot = H // Hkv, k_cache.shape[2], 0 if rope is None else rope.shape[1]

    def rotated(x, p):
        y = x.copy()
        for i in range(rot // 2):
            i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = rope[p, i], rope[p, rot // 2 + i]
            y[..., i0], y[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i1] * c + x[..., i0] * s
        return y

    for b in range(B):
        n = new_tokens(q_lens, b, T)
        for t in range(n):
            p = int(seq_lens[b]) - n + t
            if p < 0 or p >= max_len:
                continue
            for h in range(H):
                if not mask[h]:
                    q_out[b, h, t] = rotated(q[b, h, t], p + pos_offset)
            page, slot = int(page_table[b, p // page_size]), p % page_size
            for g in range(Hkv):
                keyed = not all(mask[g * group:(g + 1) * group])
                kr = rotated(k[b, g, t], p + pos_offset)
                if keyed and k_out is not None:
                    k_out[b, g, t] = kr
                if 0 <= page < k_cache.shape[0]:
                    if keyed:
                        k_cache[page, g, slot] = kr
                    v_cache[page, g, slot] = v[b, g, t]


def attend(q, k_cache, v_cache, page_table, seq_lens, q_lens, a, r, mask, max_len, prefix_table=None, prefix_len=0):
    """(o, lse, weight) of every row that has a token (NaN elsewhere): weight is
    sum_j P_j |v_j|, what the rounding of the weights can move o by."""
    B, H, T, _ = q.shape
    num_pages, Hkv, page_size, _ = k_cache.shape
    group = H // Hkv
    o, w = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full((B, H, T), np.nan)
    for b in range(B):
        n = new_tokens(q_lens, b, T)
        length = min(max(int(seq_lens[b]), 0), max_len)
        where = [(prefix_table[j // page_size], j % page_size) for j in range(prefix_len)]
        where += [(page_table[b, j // page_size], j % page_size) for j in range(length)]
        keep = np.array([j for j, (pg, _) in enumerate(where) if 0 <= pg < num_pages], dtype=np.int64)
        pages = np.array([where[j][0] for j in keep], dtype=np.int64)
        slots = np.array([where[j][1] for j in keep], dtype=np.int64)
        for h in range(H):
            kk, vv = k_cache[pages, h // group, slots], v_cache[pages, h // group, slots]
            for t in range(n):
                i = prefix_len + length - n + t
                seen = keep <= i
                j = keep[seen]
                if mask[h]:
                    s = a[h, j] + r[h, i - j]
                else:
                    s = kk[seen] @ q[b, h, t] / math.sqrt(HEAD_DIM)
                if len(s) == 0 or s.max() == -np.inf:
                    o[b, h, t], w[b, h, t], lse[b, h, t] = 0.0, 0.0, -np.inf
                    continue
                e = np.exp(s - s.max())
                lse[b, h, t] = s.max() + np.log(e.sum())
                live = e > 0
                o[b, h, t] = (e[live] / e.sum()) @ vv[seen][live]
                w[b, h, t] = (e[live] / e.sum()) @ np.abs(vv[seen][live])
    return o, lse, w
