"""Serving operators of the mixed-head layer: appending to a paged key/value cache with the position
rotation, attention of new tokens over the paged cache, and the same for a batch that shares a prefix.

Heads are of two kinds: ordinary heads attend by softmax(q.k / 8), replaced heads by the pattern
softmax(a[j] + r[i - j]); the mask says which.  With `own` false the operators run in plain torch.
"""
import math
import random

import torch

own = False

D = 64


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = {"name": name, "op": op, "B": 1, "H": 12, "Hkv": 12, "T": 1, "len": 512, "page": 64, "replaced": 3, "prefix": 0,
         "rot": 64, "interleaved": False, "k_out": False, "full": False}
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a small batch on the 12-head layer: latency
        _case("append_step_b8", "append", B=8, len=512),
        # one decode step of a large batch, shared key/value heads, small pages
        _case("append_step_b256_kv8", "append", B=256, H=32, Hkv=8, replaced=8, len=500, page=16),
        # ragged prompt chunks of odd lengths, interleaved rotation of half the columns
        _case("append_chunks_b7_t515", "append", B=7, H=12, Hkv=3, T=515, len=2050, page=32, rot=32, interleaved=True),
        # a whole prompt batch (the layer's training shape), rotated K handed to the prefill too
        _case("append_prompt_b8_t4096", "append", B=8, T=4096, len=4096, k_out=True, full=True),
        # one decode step of one short sequence: latency
        _case("decode_b1_t512", "attn", B=1, len=512, full=True),
        # an ordinary decode batch, ragged lengths
        _case("decode_b8_t4096", "attn", B=8, len=4096),
        # a large decode batch at the longest context: the cache does not fit any on-chip memory
        _case("decode_b64_t16384", "attn", B=64, len=16384, full=True),
        # five drafted tokens checked at once, shared key/value heads, small pages
        _case("draft5_b32_kv8_t8192", "attn", B=32, H=32, Hkv=8, T=5, len=8192, page=16, replaced=8),
        # a prompt chunk that continues cached sequences
        _case("chunk500_b4_t8192", "attn", B=4, H=12, Hkv=12, T=500, len=8192, page=128),
        # a few requests behind one system prompt
        _case("prefix2048_b16", "prefix", B=16, prefix=2048, len=250),
        # a batch of requests behind a long document, shared key/value heads
        _case("prefix8192_b64_kv8", "prefix", B=64, H=32, Hkv=8, replaced=8, prefix=8192, len=1000, page=16),
        # many samples of one long prompt
        _case("prefix16384_b256_kv8", "prefix", B=256, H=32, Hkv=8, replaced=8, prefix=16384, len=400),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attn", "attn", "attn", "prefix", "prefix"])
    hkv, group = rng.choice([(12, 1), (4, 1), (3, 4), (8, 4), (2, 3), (4, 8), (5, 1), (32, 1), (6, 2)])
    h = hkv * group
    c = {"op": op, "H": h, "Hkv": hkv, "page": rng.choice([16, 32, 64, 128]), "replaced": rng.choice([0, h // 4, h // 2, h // 4]),
         "prefix": 0, "rot": 64, "interleaved": False, "k_out": False, "full": rng.random() < 0.25}
    if op == "append":
        c["B"] = _log_int(rng, 1, 256)
        c["T"] = rng.choice([1, 1, 3, _log_int(rng, 2, 4096)])
        while c["B"] * c["T"] * (h + 2 * hkv) > 8 * 4096 * 36:
            if c["T"] > 1:
                c["T"] = max(1, c["T"] // 2)
            else:
                c["B"] = max(1, c["B"] // 2)
        c["len"] = c["T"] + _log_int(rng, 1, 512)
        c["rot"] = rng.choice([64, 64, 32])
        c["interleaved"] = rng.random() < 0.3
        c["k_out"] = rng.random() < 0.3
    elif op == "attn":
        c["B"] = _log_int(rng, 1, 64)
        c["T"] = rng.choice([1, 1, 1, _log_int(rng, 2, 16), _log_int(rng, 16, 500)])
        c["len"] = max(c["T"], _log_int(rng, 64, 16384))
        while c["B"] * hkv * c["len"] > 64 * 12 * 16384 or c["B"] * h * c["T"] * c["len"] > 4 * 12 * 500 * 8192:
            if c["B"] > 1:
                c["B"] //= 2
            else:
                c["T"] = max(1, c["T"] // 2)
    else:
        c["B"] = _log_int(rng, 2, 256)
        c["T"] = rng.choice([1, 1, 1, 2, 4])
        c["prefix"] = _log_int(rng, 256, 16384)
        c["len"] = max(c["T"], _log_int(rng, 8, 1000))
        while c["B"] * h * c["T"] * (c["prefix"] + c["len"]) > 256 * 32 * 16000:
            c["B"] = max(1, c["B"] // 2)
    return c


def _lens(c):
    """Tokens in the cache after this call, and new tokens, of each sequence: they belong to the case."""
    rng = random.Random("%d %d %d %d" % (c["B"], c["T"], c["len"], c["H"]))
    lens, new = [], []
    for b in range(c["B"]):
        n = c["T"] if c["full"] or c["T"] < 4 or b == 0 else rng.randint(max(1, c["T"] // 2), c["T"])
        lens.append(c["len"] if c["full"] or b == 0 else rng.randint(min(c["len"], max(n, c["len"] // 4)), c["len"]))
        new.append(n)
    return lens, new


# ------------------------------------------------------------------ state
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = random.Random(seed)
    B, H, Hkv, T, P = c["B"], c["H"], c["Hkv"], c["T"], c["page"]
    lens, new = _lens(c)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    # replaced heads spread over the layer, as a selection by score gives them
    mask = [0] * H
    for h in rng.sample(range(H), c["replaced"]):
        mask[h] = 1
    pages = [-(-n // P) for n in lens]
    prefix_pages = -(-c["prefix"] // P)
    most = max(pages)
    total = sum(pages) + prefix_pages
    order = torch.randperm(total, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    count = torch.tensor(pages, device="cuda")
    first = prefix_pages + torch.cumsum(count, 0) - count
    col = torch.arange(most, device="cuda")
    at = torch.where(col < count[:, None], first[:, None] + col, 0)
    table = torch.where(col < count[:, None], order[at], -1).to(torch.int32).contiguous()
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k_cache, v_cache = randn(total, Hkv, P, D), randn(total, Hkv, P, D)
    # slots that no token has reached yet hold whatever was in memory: NaN here
    last = torch.tensor([n - (p - 1) * P for n, p in zip(lens, pages)], device="cuda")
    stale = torch.arange(P, device="cuda") >= last[:, None]
    tail = order[first + count - 1].long()
    for cache in (k_cache, v_cache):
        cache[tail] = cache[tail].masked_fill(stale[:, None, :, None], float("nan"))
    s = {"case": c, "mask": mask, "table": table, "seq": seq, "k_cache": k_cache, "v_cache": v_cache, "max_len": max(lens),
         "new": torch.tensor(new, dtype=torch.int32, device="cuda") if min(new) < T else None}
    if c["op"] == "append":
        # q, k and v of one projection: token-major, heads side by side
        qkv = randn(B, T, H + 2 * Hkv, D).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        half = c["rot"] // 2
        angle = torch.arange(c["len"], dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(half, dtype=torch.float64, device="cuda") / half)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        s["q_out"] = torch.zeros(B, H, T, D, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16, device="cuda") if c["k_out"] else None
    else:
        s["q"] = randn(B, H, T, D)
        s["out"] = torch.zeros(B, H, T, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(B, H, T, dtype=torch.float32, device="cuda")
        n = c["prefix"] + c["len"]
        s["alpha"] = torch.randn(H, n, generator=g, device="cuda") * 0.5
        s["alpha"][:, 0] += 4.0
        s["rho"] = -0.05 * torch.arange(n, device="cuda").float() + 0.3 * torch.randn(H, n, generator=g, device="cuda")
        s["rho"][:, 0] += 2.0
        s["prefix_table"] = order[:prefix_pages].contiguous()
    s["rep"] = torch.tensor([h for h in range(H) if mask[h]], dtype=torch.int64, device="cuda")
    if own:
        from mixed_head_causal_b200 import saf
        s["mask"] = saf.head_mask(mask)
        s["kv"] = saf.PagedKV(k_cache, v_cache)
        if c["op"] != "append":
            s["workspace"] = saf.new_paged_workspace(s["kv"], B, H, T, prefix_len=c["prefix"])
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            from mixed_head_causal_b200 import saf
            saf.kv_append(s["q"], s["k"], s["v"], s["kv"], s["table"], s["seq"], mask=s["mask"], q_lens=s["new"], rope=s["rope"],
                          interleaved=c["interleaved"], max_len=s["max_len"], q_out=s["q_out"], k_out=s["k_out"])
        else:
            _append(s)
        return [s["q_out"], s["k_cache"], s["v_cache"]] + ([s["k_out"]] if c["k_out"] else [])
    if own:
        from mixed_head_causal_b200 import saf
        kw = dict(alpha=s["alpha"], rho=s["rho"], mask=s["mask"], q_lens=s["new"], max_len=s["max_len"], out=s["out"], lse=s["lse"],
                  workspace=s["workspace"])
        if c["op"] == "attn":
            return list(saf.paged_attn(s["q"], s["kv"], s["table"], s["seq"], **kw))
        return list(saf.paged_attn_prefix(s["q"], s["kv"], s["prefix_table"], c["prefix"], s["table"], s["seq"], **kw))
    return _attend(s)


def _positions(s):
    """Local position of each new token [B, T], and which of them there are."""
    T = s["case"]["T"]
    new = s["new"] if s["new"] is not None else torch.full_like(s["seq"], T)
    t = torch.arange(T, device="cuda")
    return (s["seq"] - new)[:, None] + t, t < new[:, None], new


def _rotate(x, cos, sin, rot, interleaved):
    """x [B, h, T, 64] rotated in its first `rot` columns by the angles of its tokens, in 32 bits."""
    x = x.float()
    half = rot // 2
    if interleaved:
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        x0, x1 = x[..., :half], x[..., half:rot]
    y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
    y = torch.stack([y0, y1], -1).flatten(-2) if interleaved else torch.cat([y0, y1], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def _append(s):
    c = s["case"]
    pos, there, new = _positions(s)
    angles = s["rope"][pos.clamp(0, s["rope"].shape[0] - 1)][:, None]  # [B, 1, T, rot]
    cos, sin = angles.chunk(2, -1)
    q = _rotate(s["q"], cos, sin, c["rot"], c["interleaved"])
    k = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"])
    # replaced heads have no query, and a K/V head that only they read keeps no keys
    ordinary = torch.ones(c["H"], dtype=torch.bool, device="cuda").index_fill(0, s["rep"], False)
    keyed = ordinary.view(c["Hkv"], -1).any(1)
    s["q_out"].copy_(torch.where(there[:, None, :, None] & ordinary[:, None, None], q, s["q_out"]))
    if s["k_out"] is not None:
        s["k_out"].copy_(torch.where(there[:, None, :, None] & keyed[:, None, None], k, s["k_out"]))
    # a token that is not there writes its sequence's last token again
    t = torch.minimum(torch.arange(c["T"], device="cuda"), (new - 1)[:, None]).long()
    p = pos.gather(1, t).long()
    page, slot = s["table"].gather(1, p // c["page"]).long(), p % c["page"]
    b = torch.arange(c["B"], device="cuda")[:, None]
    keep = s["k_cache"][page, :, slot]
    s["k_cache"][page, :, slot] = torch.where(keyed[:, None], k.transpose(1, 2)[b, t], keep)
    s["v_cache"][page, :, slot] = s["v"].transpose(1, 2)[b, t]


def _attend(s):
    c = s["case"]
    B, H, Hkv, T, P0 = c["B"], c["H"], c["Hkv"], c["T"], c["prefix"]
    pos, there, _ = _positions(s)
    L = s["table"].shape[1] * c["page"]
    pages = s["table"].clamp(min=0).long()
    live = torch.arange(L, device="cuda") < s["seq"][:, None]  # [B, L]
    k = s["k_cache"][pages].transpose(1, 2).reshape(B, Hkv, L, D).float()
    v = s["v_cache"][pages].transpose(1, 2).reshape(B, Hkv, L, D).float().masked_fill(~live[:, None, :, None], 0.0)
    q = s["q"].float().view(B, Hkv, -1, D)  # the group's heads and tokens are one axis
    score = (q @ k.transpose(2, 3)).view(B, H, T, L) * 0.125
    j = torch.arange(P0 + L, device="cuda")
    if P0:
        shared = s["prefix_table"].long()
        kp = s["k_cache"][shared].transpose(0, 1).reshape(Hkv, -1, D)[:, :P0].float()
        vp = s["v_cache"][shared].transpose(0, 1).reshape(Hkv, -1, D)[:, :P0].float()
        rows = q.transpose(0, 1).reshape(Hkv, -1, D)
        before = (rows @ kp.transpose(1, 2)).view(Hkv, B, H // Hkv, T, P0).transpose(0, 1).reshape(B, H, T, P0) * 0.125
        score = torch.cat([before, score], 3)
    distance = P0 + pos[:, :, None] - j  # [B, T, P0 + L]
    seen = (distance >= 0) & torch.cat([torch.ones(B, P0, dtype=torch.bool, device="cuda"), live], 1)[:, None]
    if c["replaced"]:
        rep, n = s["rep"], s["rho"].shape[1]
        score[:, rep] = (s["alpha"][rep][:, j.clamp(max=n - 1)][None, :, None]
                         + s["rho"][rep][:, distance.clamp(0, n - 1)].transpose(0, 1))
    score = score.masked_fill(~seen[:, None], float("-inf"))
    top = score.amax(3, keepdim=True)
    e = torch.exp(score - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(3, keepdim=True)
    lse = (top + torch.log(total)).squeeze(3)
    e = (e / torch.where(total == 0, 1.0, total)).view(B, Hkv, -1, P0 + L)
    o = e[..., P0:] @ v
    if P0:
        ep = e[..., :P0].transpose(0, 1).reshape(Hkv, -1, P0)
        o = o + (ep @ vp).view(Hkv, B, -1, D).transpose(0, 1)
    o = o.view(B, H, T, D).to(torch.bfloat16)
    s["out"].copy_(torch.where(there[:, None, :, None], o, s["out"]))
    s["lse"].copy_(torch.where(there[:, None], lse, s["lse"]))
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------ what a pass cannot do without
def _keyed_heads(c):
    """K/V heads that keep keys, about: a group goes keyless when all its heads are replaced."""
    group = c["H"] // c["Hkv"]
    return c["Hkv"] - (c["replaced"] if group == 1 else 0)


def work(case):
    c = case
    lens, new = _lens(c)
    H, Hkv, row = c["H"], c["Hkv"], 2 * D
    keyed, ordinary = _keyed_heads(c), c["H"] - c["replaced"]
    tokens = sum(new)
    if c["op"] == "append":
        kv = keyed + Hkv
        per_token = row * (2 * ordinary + 2 * kv + (keyed if c["k_out"] else 0))
        angles = 4 * c["rot"] * min(tokens, c["len"])
        return {"bytes": tokens * per_token + angles, "flops": tokens * 3.0 * c["rot"] * (ordinary + keyed)}
    pairs = sum(sum(c["prefix"] + n - m + t + 1 for t in range(m)) for n, m in zip(lens, new))  # (row, key) pairs of one head
    keys = c["prefix"] + sum(lens)
    moved = keys * row * (keyed + Hkv) + tokens * row * (ordinary + H) + 4 * tokens * H
    return {"bytes": moved, "flops": 2.0 * D * pairs * (2 * ordinary + c["replaced"])}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    lens, new = _lens(c)
    H, Hkv, P, P0 = c["H"], c["Hkv"], c["page"], c["prefix"]
    group = H // Hkv
    replaced = set(s["rep"].tolist())
    table = s["table"].tolist()
    if c["op"] == "append":
        half = c["rot"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
        table64 = s["rope"].double()
        q_out = s["q_out"].double()
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        k_out = torch.zeros(c["B"], Hkv, c["T"], D, dtype=torch.float64, device="cuda")

        def turn(x, p):
            turned = x.double().clone()
            z = torch.complex(turned[..., first], turned[..., second]) * torch.complex(table64[p, :half], table64[p, half:])
            turned[..., first], turned[..., second] = z.real, z.imag
            return turned

        ordinary = [h for h in range(H) if h not in replaced]
        keyed = [g for g in range(Hkv) if any(g * group + u not in replaced for u in range(group))]
        for b, (n, m) in enumerate(zip(lens, new)):
            p = torch.arange(n - m, n, device="cuda")
            pg, sl = torch.tensor(table[b], device="cuda")[p // P], p % P
            q_out[b, ordinary, :m] = turn(s["q"][b, ordinary, :m], p)
            v_cache[pg, :, sl] = s["v"][b, :, :m].transpose(0, 1).double()
            if keyed:
                kr = turn(s["k"][b, keyed, :m], p)
                k_out[b, keyed, :m] = kr
                at = torch.tensor(keyed, device="cuda")
                k_cache[pg[:, None], at, sl[:, None]] = kr.transpose(0, 1)
        return [q_out, k_cache, v_cache] + ([k_out] if c["k_out"] else [])
    out, lse = s["out"].double(), s["lse"].double()
    shared = s["prefix_table"].long()
    ks, vs = (x[shared].transpose(0, 1).reshape(Hkv, -1, D)[:, :P0].double() for x in (s["k_cache"], s["v_cache"]))
    for b, (n, m) in enumerate(zip(lens, new)):
        pg = torch.tensor(table[b][: -(-n // P)], device="cuda")
        k, v = (torch.cat([x0, x[pg].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double()], 1)
                for x0, x in ((ks, s["k_cache"]), (vs, s["v_cache"])))
        i = P0 + torch.arange(n - m, n, device="cuda")
        gap = i[:, None] - torch.arange(P0 + n, device="cuda")
        for g in range(Hkv):
            for h in range(g * group, g * group + group):
                if h in replaced:
                    z = s["alpha"][h, : P0 + n].double() + s["rho"][h].double()[gap.clamp(min=0)]
                else:
                    z = s["q"][b, h, :m].double() @ k[g].T / math.sqrt(D)
                z = torch.where(gap >= 0, z, -math.inf)
                norm = torch.logsumexp(z, 1)
                out[b, h, :m] = torch.exp(z - norm[:, None]) @ v[g]
                lse[b, h, :m] = norm
    return [out, lse]
