"""The plan of decode behind shared prefixes (host only)."""

import random

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api


def plan(lens, groups, pages, **kw):
    a = dict(num_qo_heads=8, num_kv_heads=2, page_size=16, max_pages_per_seq=4096, num_pages=10000, num_sms=152,
             host_only=True, min_shared_bytes=0)
    a.update(kw)
    return api.paged_prefix_decode_plan(lens, groups, pages, **a)


@pytest.mark.parametrize("kw,code", [
    (dict(groups=[1, 4]), L.PKA_ERR_INVALID_ARG),
    (dict(groups=[0, 3]), L.PKA_ERR_INVALID_ARG),
    (dict(groups=[0, 5]), L.PKA_ERR_INVALID_ARG),
    (dict(groups=[0, 3, 2, 4], pages=[1, 1, 1]), L.PKA_ERR_INVALID_ARG),
    (dict(pages=[-1]), L.PKA_ERR_INVALID_ARG),
    (dict(pages=[11]), L.PKA_ERR_INVALID_ARG),                        # 176 keys, a request has 170
    (dict(pages=[10], causal=True, q_len=12), L.PKA_ERR_INVALID_ARG),   # its first row sees 159
    (dict(lens=[0, 200, 200, 200], pages=[0]), L.PKA_ERR_INVALID_ARG),
    (dict(page_size=24), L.PKA_ERR_UNSUPPORTED),
    (dict(head_dim=64), L.PKA_ERR_UNSUPPORTED),
    (dict(num_qo_heads=7), L.PKA_ERR_INVALID_ARG),
    (dict(num_qo_heads=64, num_kv_heads=1, q_len=8192), L.PKA_ERR_UNSUPPORTED),   # 2^19 rows of a KV head
])
def test_refusals(kw, code):
    a = dict(lens=[170, 200, 200, 200], groups=[0, 4], pages=[4])
    a.update(kw)
    with pytest.raises(L.PkaError) as e:
        plan(**a)
    assert e.value.code == code


def test_refuses_a_window():
    d = L.DecodeDesc(batch_size=2, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, max_pages_per_seq=9,
                     num_pages=50, q_len=1, window_left=5, scale=1.0, bmm2_scale=1.0, num_sms=8,
                     flags=L.PKA_PLAN_HOST_ONLY)
    import ctypes
    i32 = lambda *x: (ctypes.c_int32 * len(x))(*x)   # noqa: E731
    h, ws = ctypes.c_void_p(), ctypes.c_size_t()
    rc = L.lib().paged_prefix_decode_plan(ctypes.byref(h), ctypes.byref(d), i32(100, 100), None, i32(0, 2), 1, i32(3), -1,
                                          ctypes.byref(ws), None)
    assert rc == L.PKA_ERR_UNSUPPORTED and not h.value


def test_binding_refuses():
    with pytest.raises(ValueError, match="one entry more"):
        plan([100, 100], [0, 2], [1, 1])
    with pytest.raises(ValueError, match="one entry more"):
        plan([100, 100], [0, 2], [1], qo_indptr=[0, 1])
    p = plan([1600] * 4, [0, 4], [90])
    with pytest.raises(ValueError, match="not made by"):
        api.paged_prefix_decode_run(api.paged_decode_plan([100], num_qo_heads=8, num_kv_heads=2, page_size=16,
                                                          max_pages_per_seq=9, num_pages=50, num_sms=8,
                                                          host_only=True), *[torch.zeros(1)] * 4)
    assert not hasattr(p, "handle")   # no other entry point takes it for its own plan


def test_groups_without_anything_to_share_are_plain_decode():
    for lens, groups, pages in (([500, 600], [0, 2], [0]), ([500, 600], [0, 1, 2], [9, 9]), ([500], [0, 0, 1], [3, 9])):
        i = plan(lens, groups, pages).info
        plain = api.paged_decode_plan(lens, num_qo_heads=8, num_kv_heads=2, page_size=16, max_pages_per_seq=4096,
                                      num_pages=10000, num_sms=152, host_only=True).info
        assert i["shared"] == 0 and i["num_prefix_pieces"] == i["num_own_pieces"] == 0
        assert all(i[k] == plain[k] for k in ("workspace_bytes", "partial_rows", "total_q", "num_sms"))


def test_little_to_share_is_plain_decode():
    """7 further requests of 2048 shared keys, 2 KV heads: 14.7 MB not read again."""
    lens, groups, pages = [2100] * 8, [0, 8], [128]
    assert plan(lens, groups, pages, min_shared_bytes=-1).info["shared"] == 0
    assert plan(lens, groups, pages, min_shared_bytes=7 * 2048 * 1024).info["shared"] == 1
    assert plan(lens, groups, pages, min_shared_bytes=7 * 2048 * 1024 + 1).info["shared"] == 0
    assert plan([8300] * 8, groups, [512], num_qo_heads=32, num_kv_heads=8, min_shared_bytes=-1).info["shared"] == 1


@pytest.mark.parametrize("seed", range(12))
def test_pieces_cover_everything_once(seed):
    """Every tile of a shared prefix for every KV head and query row, every unit behind it, each
    in one piece; partial rows that do not overlap; even shares."""
    r = random.Random(seed)
    ps, heads, kv_heads = r.choice([16, 48, 64]), 12, r.choice([1, 2, 4])
    G = heads // kv_heads
    groups, pages, lens, qo = [0], [], [], [0]
    for _ in range(r.randint(1, 6)):
        n, pre = r.randint(0, 90), r.choice([0, 1, 5, 60])
        groups.append(groups[-1] + n)
        pages.append(pre)
        for _ in range(n):
            L = r.choice([1, 1, 2, 5])
            lens.append(pre * ps + r.choice([0, 1, 16, 100, 900]) + (L if pre == 0 else 0))
            lens[-1] = max(lens[-1], L)
            qo.append(qo[-1] + L)
    if len(lens) < 2:
        lens, groups, pages, qo = [900, 901], [0, 2], [10], [0, 1, 2]
    p = plan(lens, groups, pages, num_qo_heads=heads, num_kv_heads=kv_heads, page_size=ps, qo_indptr=qo)
    i = p.info
    if not i["shared"]:
        return
    prefix, own = p.export()
    taken, tiles, units = [], {}, {}
    for row, hk, row0, lo, hi, state in prefix:
        g = groups.index(row) if groups.count(row) == 1 else max(x for x in range(len(pages)) if groups[x] == row)
        rows = (qo[groups[g + 1]] - qo[groups[g]]) * G
        assert row0 % (256) == 0 and row0 < rows and lo < hi
        taken.append((state, min(256, rows - row0)))
        for t in range(lo, hi):
            assert (g, hk, row0, t) not in tiles
            tiles[g, hk, row0, t] = 1
    want = set()
    shared = {}
    for g, pre in enumerate(pages):
        b0, b1 = groups[g], groups[g + 1]
        if b1 - b0 < 2 or pre == 0:
            continue
        rows = (qo[b1] - qo[b0]) * G
        shared.update({b: pre for b in range(b0, b1)})
        want |= {(g, hk, row0, t) for hk in range(kv_heads) for row0 in range(0, rows, 256)
                 for t in range(-(-pre * ps // 64))}
    assert set(tiles) == want
    for b, hk, row0, lo, hi, state in own:
        rows = (qo[b + 1] - qo[b]) * G
        assert row0 % 16 == 0 and row0 < rows and lo < hi
        taken.append((state, min(16, rows - row0)))
        for u in range(lo, hi):
            assert (b, hk, row0, u) not in units
            units[b, hk, row0, u] = 1
    assert set(units) == {(b, hk, row0, u) for b, n in enumerate(lens) for hk in range(kv_heads)
                          for row0 in range(0, (qo[b + 1] - qo[b]) * G, 16)
                          for u in range(shared.get(b, 0) * ps // 16, -(-n // 16))}
    at = 0
    for state, n in sorted(taken):
        assert state == at
        at += n
    assert at == i["partial_rows"] and i["workspace_bytes"] >= at * 516


def test_even_shares():
    """One prefix for 1024 rows of each of 8 KV heads, whose products bound the whole, and one for
    256, whose bytes do."""
    p = plan([65536 + 800] * 32, [0, 32], [1024], num_qo_heads=64, num_kv_heads=8, page_size=64, q_len=4,
             max_pages_per_seq=1100, num_pages=30000, causal=True)
    i = p.info
    assert i["dense"] == 1 and i["num_pairs"] == 152 and i["num_warps"] == 152 * 12
    prefix, own = p.export()
    assert sum(x[4] - x[3] for x in prefix) == 8 * 4 * 1024
    assert len(prefix) <= 152 + 32
    sizes = [x[4] - x[3] for x in own]
    assert sizes == sorted(sizes, reverse=True) and max(sizes) <= 16

    p = plan([8192 + 500] * 64, [0, 64], [512], num_qo_heads=32, num_kv_heads=8, max_pages_per_seq=600, num_pages=30000)
    i = p.info
    assert i["dense"] == 0 and i["num_pairs"] == 64 and i["num_warps"] == 152 * 12


def test_update_keeps_the_plan_where_it_refuses():
    p = plan([3000] * 8, [0, 8], [100])
    before = p.info, p.export()
    with pytest.raises(L.PkaError):
        p.update([3000] * 8, [0, 8], [190])
    with pytest.raises(L.PkaError):
        p.update([3000] * 8, [0, 7], [100])
    assert (p.info, p.export()) == before and p.batch_size == 8
    p.update([2000] * 3 + [5000] * 6, [0, 3, 9], [50, 300], qo_indptr=[0, 1, 2, 5, 6, 7, 8, 9, 10, 11])
    assert p.batch_size == 9 and p.total_q == 11 and p.info["num_prefix_pieces"] > 0
    p.update([2000, 300], [0, 1, 2], [50, 3])
    assert p.info["shared"] == 0 and p.info["num_prefix_pieces"] == 0
    p.update([3000] * 8, [0, 8], [100])
    assert (p.info, p.export()) == before
