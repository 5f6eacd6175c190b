"""What the Python serving calls refuse before anything is enqueued: tensors of the
wrong type, shape, layout or device, and sizes out of range."""
import pytest
import torch

from mixed_head_causal_b200 import saf

pytestmark = pytest.mark.gpu

B, H, HKV, T, PAGE, COLS = 2, 4, 2, 3, 16, 4


def cache():
    return saf.PagedKV(*(torch.zeros(8, HKV, PAGE, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)))


def rows(h, n=T, **kw):
    return torch.zeros(B, h, n, 64, **{"dtype": torch.bfloat16, "device": "cuda", **kw})


def ints(*shape, **kw):
    return torch.zeros(*shape, **{"dtype": torch.int32, "device": "cuda", **kw})


BAD_TABLES = {
    "table_int64": dict(page_table=lambda: ints(B, COLS, dtype=torch.int64)),
    "table_rows": dict(page_table=lambda: ints(B + 1, COLS)),
    "table_strided": dict(page_table=lambda: ints(B, 2 * COLS)[:, ::2]),
    "table_host": dict(page_table=lambda: ints(B, COLS, device="cpu")),
    "seq_length": dict(seq_lens=lambda: ints(B + 1)),
    "seq_float": dict(seq_lens=lambda: ints(B).float()),
    "q_lens_length": dict(q_lens=lambda: ints(1)),
    "max_len_large": dict(max_len=lambda: COLS * PAGE + 1),
    "max_len_past_32_bits": dict(max_len=lambda: 2 ** 32 + 5),
    "max_len_negative": dict(max_len=lambda: -1),
}


@pytest.mark.parametrize("what", [*BAD_TABLES, "k_heads", "k_type", "v_shape", "q_last_axis", "q_out_strided", "q_out_alone",
                                  "mask_length", "rope_type", "offset", "offset_negative", "k_out_shape"])
def test_append_refuses(what):
    f = dict(q=lambda: rows(H), k=lambda: rows(HKV), v=lambda: rows(HKV), page_table=lambda: ints(B, COLS),
             seq_lens=lambda: ints(B))
    f.update(BAD_TABLES.get(what) or {
        "k_heads": dict(k=lambda: rows(HKV + 1)), "k_type": dict(k=lambda: rows(HKV, dtype=torch.float16)),
        "v_shape": dict(v=lambda: rows(HKV, T + 1)), "q_last_axis": dict(q=lambda: rows(H).transpose(2, 3).contiguous().transpose(2, 3)),
        "q_out_strided": dict(q_out=lambda: rows(2 * H)[:, ::2]), "q_out_alone": dict(q=lambda: None, q_out=lambda: rows(H)),
        "mask_length": dict(mask=lambda: [0] * (H + 1)), "rope_type": dict(rope=lambda: torch.zeros(80, 64, device="cuda").double()),
        "offset": dict(pos_offset=lambda: 2 ** 32), "offset_negative": dict(pos_offset=lambda: -1),
        "k_out_shape": dict(k_out=lambda: rows(H))}[what])
    a = {n: x() for n, x in f.items()}
    with pytest.raises(ValueError):
        saf.kv_append(a.pop("q"), a.pop("k"), a.pop("v"), cache(), a.pop("page_table"), a.pop("seq_lens"), **a)


@pytest.mark.parametrize("prefix", [0, 20])
@pytest.mark.parametrize("what", [*BAD_TABLES, "q_strided", "q_type", "q_width", "mask_length", "no_pattern", "pattern_heads",
                                  "pattern_type", "out_shape", "lse_type", "workspace_host"])
def test_attention_refuses(what, prefix):
    f = dict(q=lambda: rows(H), page_table=lambda: ints(B, COLS), seq_lens=lambda: ints(B))
    pat = lambda h=H, **kw: torch.zeros(h, 200, **{"device": "cuda", **kw})
    f.update(BAD_TABLES.get(what) or {
        "q_strided": dict(q=lambda: rows(2 * H)[:, ::2]), "q_type": dict(q=lambda: rows(H).float()),
        "q_width": dict(q=lambda: torch.cat([rows(H)] * 2, 3)), "mask_length": dict(mask=lambda: [0] * (H - 1)),
        "no_pattern": dict(mask=lambda: [0, 1, 0, 0]),
        "pattern_heads": dict(mask=lambda: [0, 1, 0, 0], alpha=pat, rho=lambda: pat(H - 1)),
        "pattern_type": dict(mask=lambda: [0, 1, 0, 0], alpha=lambda: pat().bfloat16(), rho=pat),
        "out_shape": dict(out=lambda: rows(H, T + 1)), "lse_type": dict(lse=lambda: torch.zeros(B, H, T, device="cuda").half()),
        "workspace_host": dict(workspace=lambda: torch.zeros(1 << 20, dtype=torch.uint8))}[what])
    a = {n: x() for n, x in f.items()}
    q, table, seq = a.pop("q"), a.pop("page_table"), a.pop("seq_lens")
    with pytest.raises(ValueError):
        if prefix:
            saf.paged_attn_prefix(q, cache(), ints(2), prefix, table, seq, **a)
        else:
            saf.paged_attn(q, cache(), table, seq, **a)


def test_library_refusals_reach_python():
    """What the library itself refuses comes as SafError: a small or misaligned workspace, a short pattern."""
    q, table, seq, kv = rows(H), ints(B, COLS), ints(B), cache()
    ws = saf.new_paged_workspace(kv, B, H, T)
    pat = torch.zeros(H, COLS * PAGE - 1, device="cuda")
    for kw in (dict(workspace=ws[:-1]), dict(workspace=torch.zeros(ws.numel() + 256, dtype=torch.uint8, device="cuda")[8:]),
               dict(mask=[0, 1, 0, 0], alpha=pat, rho=pat)):
        with pytest.raises(saf.SafError):
            saf.paged_attn(q, kv, table, seq, **kw)
    for prefix, n in ((20, 1), (20, 3), (-1, 0), (2 ** 32 + 1, 1)):
        with pytest.raises((ValueError, saf.SafError)):
            saf.paged_attn_prefix(q, kv, ints(n), prefix, table, seq)


def test_cache_refusals():
    k = torch.zeros(4, HKV, PAGE, 64, dtype=torch.bfloat16, device="cuda")
    for a, b in ((k.half(), k.half()), (k, k[:2]), (k[..., :32], k[..., :32]), (k.transpose(2, 3), k.transpose(2, 3)), (k, k.cpu()),
                 (k[0], k[0])):
        with pytest.raises(ValueError):
            saf.PagedKV(a, b)
    odd = saf.PagedKV(*(torch.zeros(4, HKV, 24, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    none = saf.PagedKV(*(torch.zeros(0, HKV, PAGE, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    for kv in (odd, none, saf.PagedKV(k[:, :1].expand(4, HKV, PAGE, 64), k)):    # (the last: heads one on the other)
        with pytest.raises(saf.SafError):
            saf.paged_attn(rows(H), kv, ints(B, COLS), ints(B))
