"""Latent attention on the GPU against the plain 64-bit form: page tables and slot maps,
cache rows, absorbed decode, expanded prefill, and a run of them together."""
import math
import random

import pytest
import torch

from latent_ref import (assert_within, ref_decode, ref_prefill, ref_tables)
from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---- page tables -------------------------------------------------------------------

def tables_case(kv, new, ps, num_slots, width=None, spare=5, head=2, seed=0):
    r = random.Random(seed)
    width = width or max(1, max(-(-(n + w) // ps) for n, w in zip(kv, new)))
    pool = sum(-(-(n + w) // ps) for n, w in zip(kv, new)) + spare
    perm = list(range(pool))
    r.shuffle(perm)
    table, at = [], 0
    for n in kv:
        have = -(-n // ps)
        table.append(perm[at:at + have] + [-1] * (width - have))
        at += have
    return table, [-7] * head + perm[at:], head, num_slots


def run_tables(kv, new, table, free, head, ps, num_slots):
    tab = i32(table)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    res = api.paged_kv_tables(i32(kv), i32(new), i32(free), i32([head]), tab, page_size=ps,
                              num_slots=num_slots, status=status)
    return tab, res, status


@pytest.mark.parametrize("kv,new,ps,slots", [
    ([0], [1], 16, 1),
    ([0, 15, 16, 17], [1, 1, 1, 1], 16, 4),
    ([5, 0, 0, 33], [0, 0, 40, 7], 8, 100),
    ([0, 0, 0], [0, 0, 0], 32, 3),
    ([100] * 700, [3] * 700, 48, 2100),
    (list(range(1500)), [i % 5 for i in range(1500)], 1, 3100),
    ([7, 0], [4000, 1], 64, 5000),
])
def test_tables_follow_the_plain_form(kv, new, ps, slots):
    table, free, head, slots = tables_case(kv, new, ps, slots)
    want = ref_tables(kv, new, free, head, table, ps, slots)
    tab, res, status = run_tables(kv, new, table, free, head, ps, slots)
    api.check_status(status)
    assert tab.tolist() == want[0]
    assert res.seq_lens.tolist() == want[1]
    assert res.qo_indptr.tolist() == want[2]
    assert res.slot_map.tolist() == want[3]
    assert res.free_head.tolist() == [want[4]]


def test_tables_of_the_largest_batch():
    B, ps = 16384, 16
    r = random.Random(4)
    kv = [r.choice([0, 1, 15, 16, 40]) for _ in range(B)]
    new = [r.choice([0, 1, 1, 17]) for _ in range(B)]
    table, free, head, slots = tables_case(kv, new, ps, sum(new) + 100)
    want = ref_tables(kv, new, free, head, table, ps, slots)
    tab, res, status = run_tables(kv, new, table, free, head, ps, slots)
    api.check_status(status)
    assert tab.tolist() == want[0] and res.slot_map.tolist() == want[3]
    assert res.qo_indptr.tolist() == want[2] and res.free_head.tolist() == [want[4]]


def test_tables_slots_past_32_bits():
    table, ps = [[2 ** 31 - 1, -1]], 65536
    tab, res, _ = run_tables([65535], [2], table, [2 ** 31 - 2], 0, ps, 2)
    assert res.slot_map.tolist() == [(2 ** 31 - 1) * ps + 65535, (2 ** 31 - 2) * ps]
    assert tab.tolist() == [[2 ** 31 - 1, 2 ** 31 - 2]]


@pytest.mark.parametrize("kv,new,slots,width,free_n,head", [
    ([10, 3], [40, 1], 60, 3, 9, 0),        # a row of the table is too short
    ([10, 3], [20, 1], 20, 4, 9, 0),        # more tokens than slots
    ([10, 3], [20, 30], 60, 4, 2, 0),       # too few pages
    ([10, 3], [20, 30], 60, 4, 9, 7),       # too few pages behind the head: 3 wanted, 2 left
    ([10, -1], [20, 3], 60, 4, 9, 0),       # a negative length
    ([10, 3], [20, -3], 60, 4, 9, 0),
    ([10, 3], [20, 3], 60, 4, 9, -1),       # a negative head
])
def test_tables_step_that_does_not_fit_changes_nothing(kv, new, slots, width, free_n, head):
    table = [[100 + 10 * b + j if j < -(-max(n, 0) // 16) else -1 for j in range(width)]
             for b, n in enumerate(kv)]
    tab, res, status = run_tables(kv, new, table, list(range(free_n)), head, 16, slots)
    with pytest.raises(L.PkaError) as e:
        api.check_status(status)
    assert e.value.code == L.PKA_ERR_DEVICE_CAPACITY
    api.check_status(status)   # reading it cleared it
    assert tab.tolist() == table
    assert res.seq_lens.tolist() == kv
    assert res.qo_indptr.tolist() == [0] * (len(kv) + 1)
    assert res.slot_map.tolist() == [-1] * slots
    assert res.free_head.tolist() == [head]


def test_tables_step_that_takes_the_last_free_page():
    kv, new = [10, 3], [20, 30]          # one page and two
    table, free = [[100, -1, -1, -1], [110, -1, -1, -1]], list(range(9))
    tab, res, status = run_tables(kv, new, table, free, 6, 16, 60)
    api.check_status(status)
    want = ref_tables(kv, new, free, 6, table, 16, 60)
    assert tab.tolist() == want[0] and res.slot_map.tolist() == want[3]
    assert res.free_head.tolist() == [9]


def test_tables_rejects_overlapping_and_misplaced_arguments():
    kv, new, free = i32([3, 4]), i32([1, 1]), i32([5, 6])
    tab, head = i32([[1, -1], [2, -1]]), i32([0])
    kw = dict(page_size=16, num_slots=2)
    with pytest.raises(L.PkaError, match="overlaps"):
        api.paged_kv_tables(kv, new, free, head, tab, seq_lens=kv, **kw)
    with pytest.raises(L.PkaError, match="overlaps"):
        api.paged_kv_tables(kv, new, free, head, tab, free_head_out=head, **kw)
    with pytest.raises(L.PkaError, match="overlap"):
        api.paged_kv_tables(kv, new, free, head, tab, status=kv[:1], **kw)
    with pytest.raises(ValueError, match="cpu"):
        api.paged_kv_tables(kv.cpu(), new, free, head, tab, **kw)
    with pytest.raises(ValueError, match="int32"):
        api.paged_kv_tables(kv.long(), new, free, head, tab, **kw)
    with pytest.raises(ValueError, match="one row per request"):
        api.paged_kv_tables(kv, new[:1], free, head, tab, **kw)
    big = torch.zeros(16385, dtype=torch.int32, device=DEV)
    with pytest.raises(L.PkaError) as e:
        api.paged_kv_tables(big, big.clone(), free, head, big.view(-1, 1).clone(), **kw)
    assert e.value.code == L.PKA_ERR_UNSUPPORTED


# ---- cache rows --------------------------------------------------------------------

@pytest.mark.parametrize("tokens,dl,dr,ps,dtype", [
    (1, 512, 64, 16, BF), (33, 256, 64, 8, HF), (1000, 512, 64, 48, BF), (7, 8, 8, 3, HF),
    (5, 72, 0, 1, BF), (9001, 512, 64, 16, BF), (8193, 2048, 512, 7, HF), (3, 4096, 8, 2, BF)])
def test_append_writes_rows_and_nothing_else(tokens, dl, dr, ps, dtype):
    g = torch.Generator(device=DEV).manual_seed(3)
    n_pages = tokens // ps + 4
    D = dl + dr
    wide = torch.randn((n_pages, ps + 2, D), generator=g, device=DEV).to(dtype)
    pages = wide[:, :ps]                                   # pages with a gap behind them
    rows = torch.randn((tokens, 8 + D + 16), generator=g, device=DEV).to(dtype)
    latent, rope = rows[:, 8:8 + dl], rows[:, 8 + dl:8 + D] if dr else None
    slots = torch.randperm(n_pages * ps, generator=torch.Generator().manual_seed(1))[:tokens]
    slots = slots.to(DEV)
    if tokens > 2:
        slots[tokens // 2] = -1
    want = wide.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[s // ps, s % ps] = rows[t, 8:8 + D]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = api.paged_latent_append(latent, rope, slots, pages, status=status)
    api.check_status(status)
    assert got is pages
    assert torch.equal(wide, want)


def test_append_skips_and_reports_slots_past_the_pool():
    pages = torch.zeros((2, 8, 64), dtype=BF, device=DEV)
    rows = torch.ones((4, 64), dtype=BF, device=DEV)
    slots = torch.tensor([3, 16, 2 ** 40, -2 ** 40], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    api.paged_latent_append(rows, None, slots, pages, status=status)
    with pytest.raises(L.PkaError) as e:
        api.check_status(status)
    assert e.value.code == L.PKA_ERR_DEVICE_BOUNDS
    assert float(pages.float().sum()) == 64 and float(pages[0, 3].float().sum()) == 64
    api.paged_latent_append(rows, None, slots, pages)        # without a status word
    api.paged_latent_append(rows[:0], None, slots[:0], pages)
    torch.cuda.synchronize()


def test_append_offsets_past_32_bits():
    ps, D = 64, 576
    n_pages = 2 ** 32 // (ps * D) + 3                        # elements and bytes pass 2^32
    pages = torch.zeros((n_pages, ps, D), dtype=BF, device=DEV)
    rows = torch.randn((2, D), device=DEV).to(BF)
    slots = torch.tensor([n_pages * ps - 1, 5], device=DEV)
    api.paged_latent_append(rows[:, :512], rows[:, 512:], slots, pages)
    assert torch.equal(pages[-1, -1], rows[0]) and torch.equal(pages[0, 5], rows[1])


# ---- absorbed decode ---------------------------------------------------------------

def decode_inputs(kv_lens, qo, heads, dl, ps, dtype, seed=0, junk=float("nan"), pool_slack=3):
    """Pages that hold ``junk`` wherever no token lies, tables with -1 behind a request."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-n // ps) for n in kv_lens]
    pool, D = sum(need) + pool_slack, dl + 64
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    pages = torch.full((pool, ps, D), junk, dtype=dtype, device=DEV)
    width = max(1, max(need)) + 1
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(kv_lens):
        ids = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = torch.tensor(ids, dtype=torch.int32)
        if n:
            flat = torch.full((need[b] * ps, D), junk, dtype=dtype, device=DEV)
            flat[:n] = torch.randn((n, D), generator=g, device=DEV).to(dtype)
            pages[torch.tensor(ids, device=DEV)] = flat.view(need[b], ps, D)
    q = torch.randn((qo[-1], heads, D), generator=g, device=DEV).to(dtype)
    return q, pages, table.to(DEV)


def check_decode(kv_lens, q_lens, heads, dl=512, ps=16, dtype=BF, out_dtype=None, causal=False,
                 scale=None, out_scale=1.0, live=None, num_sms=0, seed=0, packed=False):
    qo = [0]
    for n in q_lens:
        qo.append(qo[-1] + n)
    q, pages, table = decode_inputs(kv_lens, qo, heads, dl, ps, dtype, seed)
    scale = 1 / math.sqrt(dl + 64) if scale is None else scale
    kw = dict(qo_indptr=qo) if packed else dict(q_len=q_lens[0])
    plan = api.paged_latent_decode_plan(
        kv_lens, num_heads=heads, page_size=ps, max_pages_per_seq=table.shape[1],
        num_pages=pages.shape[0], scale=scale, latent_dim=dl, causal=causal,
        output_scale=out_scale, return_lse=True, freeze_seq_lens=live is None, num_sms=num_sms,
        dtype=dtype, out_dtype=out_dtype, **kw)
    out, lse = api.paged_latent_decode_run(plan, q, pages, table,
                                           seq_lens_kv=None if live is None else i32(live))
    plan.check()
    ref = ref_decode(q, pages, table, kv_lens if live is None else live, qo, dl, scale, causal,
                     out_scale, out.dtype)
    assert_within(out, lse, ref)
    return plan, out, lse


@pytest.mark.parametrize("heads", [1, 5, 8, 16, 17, 32, 40, 64, 65, 128])
@pytest.mark.parametrize("dl", [256, 512])
def test_decode_heads(heads, dl):
    check_decode([1, 63, 64, 65, 700], [1] * 5, heads, dl=dl)


@pytest.mark.parametrize("ps", [8, 16, 24, 32, 48, 64, 128, 200, 256])
def test_decode_page_sizes(ps):
    check_decode([1, ps - 1, ps, ps + 1, 5 * ps + 3, 777], [1] * 6, 16, ps=ps, seed=ps)


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, FP), (BF, HF), (HF, HF), (HF, BF), (HF, FP)])
def test_decode_types(dtype, out_dtype):
    check_decode([300, 40, 129], [1] * 3, 24, dtype=dtype, out_dtype=out_dtype, dl=256,
                 out_scale=0.75)


@pytest.mark.parametrize("heads", [4, 16, 32, 64])
def test_decode_causal_rows(heads):
    check_decode([3, 64, 66, 500, 129], [3] * 5, heads, causal=True)


def test_decode_packed_rows_and_requests_without_rows():
    check_decode([70, 0, 10, 200, 5], [2, 1, 0, 5, 1], 12, causal=True, packed=True)
    check_decode([70, 0, 10, 200, 5], [2, 1, 0, 5, 1], 40, causal=False, packed=True, dl=256)


def test_decode_rows_that_see_nothing():
    # more causal rows than keys, and requests without keys: zeros and -inf
    plan, out, lse = check_decode([0, 2, 1, 130], [4] * 4, 20, causal=True)
    assert bool((out[:4] == 0).all()) and bool((lse[:6] == -math.inf).all())


@pytest.mark.parametrize("num_sms", [1, 3, 16, 152])
@pytest.mark.parametrize("heads,dl", [(8, 512), (64, 512), (128, 256)])
def test_decode_split_over_the_length(num_sms, heads, dl):
    plan, _, _ = check_decode([5000, 0, 1, 700, 64 * 30], [1] * 5, heads, dl=dl, ps=32,
                              num_sms=num_sms, seed=num_sms)
    if num_sms >= 16:
        assert plan.info["num_split"] >= 1


@pytest.mark.parametrize("dl", [256, 512])
@pytest.mark.parametrize("batch,heads", [(1, 16), (5, 64), (24, 64), (3, 128), (24, 100)])
def test_decode_requests_of_many_pieces(batch, heads, dl):
    """Few and many rows of ten pieces and more: the merge shares them out differently."""
    plan, _, _ = check_decode([2600 + 64 * b for b in range(batch)], [1] * batch, heads, dl=dl,
                              num_sms=min(1024, 20 * batch * (2 if heads > 64 else 1)))
    assert plan.info["num_split"] == batch and plan.info["num_items"] >= 9 * batch


@pytest.mark.parametrize("live", [[2000, 5, 64], [1, 0, 63], [1999, 900, 0], [640, 128, 1]])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_decode_live_lengths(live, heads):
    check_decode([2000, 900, 64], [1] * 3, heads, live=live)


def test_decode_live_lengths_outside_the_plan_are_clamped():
    q, pages, table = decode_inputs([100, 100], [0, 1, 2], 16, 512, 16, BF)
    plan = api.paged_latent_decode_plan([100, 100], num_heads=16, page_size=16, scale=0.04,
                                        max_pages_per_seq=table.shape[1], return_lse=True,
                                        num_pages=pages.shape[0], freeze_seq_lens=False)
    out, lse = api.paged_latent_decode_run(plan, q, pages, table, seq_lens_kv=i32([2 ** 31 - 1, -5]))
    plan.check()
    assert_within(out, lse, ref_decode(q, pages, table, [100, 0], [0, 1, 2], 512, 0.04, False, 1.0, BF))


@pytest.mark.parametrize("heads", [16, 64])   # 32 and 128 rows a request
@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 40.0])
def test_decode_scales(scale, heads):
    check_decode([1, 300, 77], [2] * 3, heads, scale=scale, causal=True, dl=256)


@pytest.mark.parametrize("heads,q_lens,dtype,out_dtype,dl,ps", [
    (40, [2, 2, 2], BF, FP, 512, 8),          # 80 rows: the second CTA of a pair nearly empty
    (33, [4, 4, 4], HF, BF, 256, 24),         # queries by plain loads, 132 rows: two row blocks
    (130, [1, 1, 1], HF, HF, 512, 32),
    (128, [3, 3, 3], BF, BF, 512, 256),       # three row blocks
    (1024, [1, 1, 1], BF, HF, 256, 16),
])
def test_decode_many_rows(heads, q_lens, dtype, out_dtype, dl, ps):
    check_decode([500, 63, 1], q_lens, heads, dl=dl, ps=ps, dtype=dtype, out_dtype=out_dtype,
                 causal=True, out_scale=0.5)
    check_decode([500, 64, 0], q_lens, heads, dl=dl, ps=ps, dtype=dtype, out_dtype=out_dtype,
                 live=[401, 1, 0], num_sms=20)


@pytest.mark.parametrize("heads", [16, 48, 100])
def test_decode_growing_scores_rescale_the_output(heads):
    """Each key tile's scores tower over the last one's, so that every tile moves the
    running maximum and rescales what was summed before."""
    kv, dl = [1500], 512
    q, pages, table = decode_inputs(kv, [0, 1], heads, dl, 16, BF)
    d = torch.randn(dl + 64, device=DEV)
    d /= d.norm()
    q = (d * 20 + torch.randn((1, heads, dl + 64), device=DEV) * 0.1).to(BF)
    ids = table[0, :94].long()
    flat = pages[ids].flatten(0, 1).float()
    flat[:1500] += d * (torch.arange(1500, device=DEV)[:, None] * 0.05)
    pages[ids] = flat.to(BF).view(94, 16, -1)
    for sms in (1, 8):
        plan = api.paged_latent_decode_plan(kv, num_heads=heads, page_size=16, scale=0.5,
                                            max_pages_per_seq=table.shape[1], num_sms=sms,
                                            num_pages=pages.shape[0], return_lse=True)
        out, lse = api.paged_latent_decode_run(plan, q, pages, table)
        plan.check()
        assert_within(out, lse, ref_decode(q, pages, table, kv, [0, 1], dl, 0.5, False, 1.0, BF))


@pytest.mark.parametrize("heads", [12, 24, 70, 72])
def test_decode_strided_arguments_and_rows_behind_the_batch(heads):
    kv, dl, D = [90, 200], 256, 320
    q, pages, table = decode_inputs(kv, [0, 1, 2], heads, dl, 16, HF)
    qw = torch.zeros((4, heads, 3, D), dtype=HF, device=DEV)
    qw[:2, :, 1] = q
    pw = torch.full((pages.shape[0], 20, D), float("nan"), dtype=HF, device=DEV)
    pw[:, :16] = pages
    tw = torch.full((2, table.shape[1] + 5), 10 ** 9, dtype=torch.int32, device=DEV)
    tw[:, :table.shape[1]] = table
    plan = api.paged_latent_decode_plan(kv, num_heads=heads, page_size=16, scale=0.05,
                                        max_pages_per_seq=table.shape[1], latent_dim=dl,
                                        num_pages=pages.shape[0], return_lse=True, dtype=HF)
    out = torch.full((4, heads, dl), 7.0, dtype=HF, device=DEV)
    lse = torch.full((4, heads), 7.0, device=DEV)
    api.paged_latent_decode_run(plan, qw[:, :, 1], pw[:, :16], tw, out=out, lse=lse)
    plan.check()
    assert_within(out[:2], lse[:2], ref_decode(q, pages, table, kv, [0, 1, 2], dl, 0.05, False,
                                               1.0, HF))
    assert bool((out[2:] == 7).all()) and bool((lse[2:] == 7).all())


@pytest.mark.parametrize("heads", [16, 80])
def test_decode_bad_pages_read_as_zeros(heads):
    q, pages, table = decode_inputs([64, 64], [0, 1, 2], heads, 256, 16, BF, junk=0.0)
    clean = table.clone()
    table[0, 1], table[1, 2] = pages.shape[0], -3
    plan = api.paged_latent_decode_plan([64, 64], num_heads=heads, page_size=16, scale=0.05,
                                        max_pages_per_seq=table.shape[1], latent_dim=256,
                                        num_pages=pages.shape[0], return_lse=True)
    out, lse = api.paged_latent_decode_run(plan, q, pages, table)
    plan.check()
    zeroed = torch.cat([pages, torch.zeros_like(pages[:1])])
    clean[0, 1] = clean[1, 2] = pages.shape[0]
    assert_within(out, lse, ref_decode(q, zeroed, clean, [64, 64], [0, 1, 2], 256, 0.05, False,
                                       1.0, BF))


@pytest.mark.parametrize("num_sms", [1, 8])      # whole and cut requests
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_decode_nan_in_a_cached_row_reaches_its_own_request_only(heads, num_sms):
    """Output and LSE of the request are NaN, also where only one of its pieces has
    the row; other requests, in the same CTAs before and behind it, are as ever."""
    kv = [300, 700, 65, 500]
    q, pages, table = decode_inputs(kv, list(range(5)), heads, 256, 16, BF)
    plan = api.paged_latent_decode_plan(kv, num_heads=heads, page_size=16, scale=0.05,
                                        max_pages_per_seq=table.shape[1], num_pages=pages.shape[0],
                                        latent_dim=256, return_lse=True, num_sms=num_sms)
    assert (plan.info["num_split"] >= 1) == (num_sms > 1)
    good, good_lse = api.paged_latent_decode_run(plan, q, pages, table)
    pages[int(table[1, 40]), 3, 7] = float("nan")     # token 643 of request 1
    out, lse = api.paged_latent_decode_run(plan, q, pages, table)
    plan.check()
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
    for b in (0, 2, 3):
        assert bool(good[b].isfinite().all())
        assert torch.equal(out[b], good[b]) and torch.equal(lse[b], good_lse[b])


@pytest.mark.parametrize("heads,dl", [(64, 512), (128, 512), (128, 256)])
def test_decode_bad_pages_far_into_a_request_read_as_zeros(heads, dl):
    """Entries outside the pool in tiles that are asked for ahead of their copies."""
    kv = [1000, 640]
    q, pages, table = decode_inputs(kv, [0, 1, 2], heads, dl, 16, BF)
    plan = api.paged_latent_decode_plan(kv, num_heads=heads, page_size=16, scale=0.05,
                                        max_pages_per_seq=table.shape[1], num_pages=pages.shape[0],
                                        latent_dim=dl, num_sms=2, return_lse=True)
    bad = [(0, 20, -1), (0, 33, pages.shape[0]), (0, 50, 2 ** 31 - 1), (1, 30, -2 ** 31)]
    rows = torch.zeros((len(bad), 16, dl + 64), dtype=BF, device=DEV)
    fixed, pool = table.clone(), torch.cat([pages, rows])
    for i, (b, j, entry) in enumerate(bad):
        table[b, j] = entry
        fixed[b, j] = pages.shape[0] + i
    out, lse = api.paged_latent_decode_run(plan, q, pages, table)
    plan.check()
    ref = ref_decode(q, pool, fixed, kv, [0, 1, 2], dl, 0.05, False, 1.0, BF)
    assert_within(out, lse, ref)


@pytest.mark.parametrize("heads", [16, 128])
def test_decode_pool_offsets_past_32_bits(heads):
    ps, D = 64, 576
    n_pages = 2 ** 32 // (ps * D) + 10
    pages = torch.full((n_pages, ps, D), float("nan"), dtype=BF, device=DEV)
    ids = [n_pages - 1, 3, n_pages - 2]
    for p in ids:
        pages[p] = torch.randn((ps, D), device=DEV).to(BF)
    table = i32([ids])
    q = torch.randn((1, heads, D), device=DEV).to(BF)
    plan = api.paged_latent_decode_plan([180], num_heads=heads, page_size=ps, max_pages_per_seq=3,
                                        num_pages=n_pages, scale=0.04, return_lse=True)
    out, lse = api.paged_latent_decode_run(plan, q, pages, table)
    plan.check()
    assert_within(out, lse, ref_decode(q, pages, table, [180], [0, 1], 512, 0.04, False, 1.0, BF))


@pytest.mark.parametrize("heads", [32, 128])
def test_decode_gives_the_same_bits_again_and_in_two_streams(heads):
    kv = [4000, 17, 900]
    q, pages, table = decode_inputs(kv, [0, 1, 2, 3], heads, 512, 16, BF)
    plan = api.paged_latent_decode_plan(kv, num_heads=heads, page_size=16, scale=0.04,
                                        max_pages_per_seq=table.shape[1],
                                        num_pages=pages.shape[0], return_lse=True)
    first = api.paged_latent_decode_run(plan, q, pages, table)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(api.paged_latent_decode_run(plan, q, pages, table))
    torch.cuda.synchronize()
    plan.check()
    for out, lse in got:
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("heads", [16, 128])
def test_decode_split_requests_captured_and_on_a_given_stream(heads):
    """The decode and the merge behind it, captured; replays on other lengths; and the same
    call on a stream that is not the current one, its workspace made and freed there."""
    kv = [6000, 40, 3000]
    q, pages, table = decode_inputs(kv, [0, 1, 2, 3], heads, 512, 16, BF)
    plan = api.paged_latent_decode_plan(kv, num_heads=heads, page_size=16, scale=0.04,
                                        max_pages_per_seq=table.shape[1], return_lse=True,
                                        num_pages=pages.shape[0], freeze_seq_lens=False)
    assert plan.info["num_split"] >= 2
    lens, out = i32(kv), torch.empty((3, heads, 512), dtype=BF, device=DEV)
    lse = torch.empty((3, heads), device=DEV)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_latent_decode_run(plan, q, pages, table, seq_lens_kv=lens, out=out, lse=lse,
                                    workspace=ws)
    for now in (kv, [100, 0, 2999], [5999, 17, 1]):
        lens.copy_(i32(now))
        out.fill_(float("nan"))
        graph.replay()
        plan.check()
        ref = ref_decode(q, pages, table, now, [0, 1, 2, 3], 512, 0.04, False, 1.0, BF)
        assert_within(out, lse, ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = api.paged_latent_decode_run(plan, q, pages, table, seq_lens_kv=lens, stream=stream)
        torch.full((plan.workspace_bytes // 4,), float("nan"), device=DEV)   # not the call's memory
        side.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_decode_plan_update_and_refusals():
    kv = [300, 40]
    q, pages, table = decode_inputs([300, 40, 999], [0, 1, 2, 3], 16, 256, 16, BF)
    args = dict(num_heads=16, page_size=16, max_pages_per_seq=table.shape[1], scale=0.05,
                num_pages=pages.shape[0], latent_dim=256, return_lse=True)
    plan = api.paged_latent_decode_plan(kv, **args)
    plan.update([300, 40, 999])
    out, lse = api.paged_latent_decode_run(plan, q, pages, table)
    plan.check()
    assert_within(out, lse, ref_decode(q, pages, table, [300, 40, 999], [0, 1, 2, 3], 256, 0.05,
                                       False, 1.0, BF))
    run = api.paged_latent_decode_run
    for bad, what in [(dict(q=q[:2]), "q must be"), (dict(q=q.half()), "bfloat16"),
                      (dict(q=q.cpu()), "cpu"), (dict(pages=pages[1:]), "pages must be"),
                      (dict(block_tables=table[:, :-1]), "max_pages_per_seq"),
                      (dict(block_tables=table.long()), "int32"),
                      (dict(out=torch.zeros_like(q[..., :128])), "contiguous|out must"),
                      (dict(lse=torch.zeros((3, 15), device=DEV)), "lse must")]:
        with pytest.raises(ValueError, match=what):
            run(plan, **{**dict(q=q, pages=pages, block_tables=table), **bad})
    big = api.paged_latent_decode_plan([300, 40, 999], num_sms=152, **args)
    if big.workspace_bytes:
        with pytest.raises(L.PkaError) as e:
            run(big, q, pages, table, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
        assert e.value.code == L.PKA_ERR_WORKSPACE_TOO_SMALL
    live = api.paged_latent_decode_plan(kv, freeze_seq_lens=False, **args)
    with pytest.raises(L.PkaError, match="seq_lens_kv_dev"):
        run(live, q, pages, table)


# ---- expanded prefill ----------------------------------------------------------------

def check_prefill(lq, lk, heads, causal=True, dtype=BF, out_dtype=None, scale=None, out_scale=1.0,
                  seed=0, rows=None, fused=True, num_sms=0, cut=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qo, ko = [0], [0]
    for a, b in zip(lq, lk):
        qo.append(qo[-1] + a)
        ko.append(ko[-1] + b)
    q = torch.randn((qo[-1], heads, 192), generator=g, device=DEV).to(dtype)
    kv = torch.randn((ko[-1], heads, 256), generator=g, device=DEV).to(dtype)
    k, v = (kv[..., :128], kv[..., 128:]) if fused else (kv[..., :128].contiguous(),
                                                         kv[..., 128:].contiguous())
    rope = torch.randn((ko[-1], 96), generator=g, device=DEV).to(dtype)[:, 16:80]
    plan = api.batch_latent_prefill_plan(qo, ko, num_heads=heads, causal=causal, sm_scale=scale,
                                         output_scale=out_scale, return_lse=True, dtype=dtype,
                                         out_dtype=out_dtype, num_sms=num_sms)
    assert cut is None or (plan.workspace_bytes > 0) == cut
    out, lse = api.batch_latent_prefill_run(plan, q, k, rope, v)
    plan.check()
    scale = 192 ** -0.5 if scale is None else scale
    picked, ref = ref_prefill(q, k, rope, v, qo, ko, scale, causal, out_scale, out.dtype, rows)
    assert_within(out[picked], lse[picked], ref)
    return out, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([1, 64, 65, 127], [1, 64, 65, 127]),
                                   ([128, 129, 3], [200, 129, 300]), ([0, 5, 0], [0, 70, 4])])
def test_prefill_lengths(lq, lk, causal):
    check_prefill(lq, lk, 3, causal)


@pytest.mark.parametrize("dtype,out_dtype", [(BF, FP), (BF, HF), (HF, HF), (HF, FP), (HF, BF)])
def test_prefill_types(dtype, out_dtype):
    check_prefill([70, 33], [90, 200], 2, dtype=dtype, out_dtype=out_dtype, out_scale=0.5,
                  fused=False)


@pytest.mark.parametrize("scale", [0.0, 0.3, 3.0])
def test_prefill_scales(scale):
    check_prefill([100], [150], 2, scale=scale)


@pytest.mark.parametrize("num_sms,cut", [(1, False), (2, False), (16, True), (152, True)])
@pytest.mark.parametrize("causal,dtype,out_dtype", [(True, BF, BF), (False, HF, FP), (True, HF, BF)])
def test_prefill_tiles_cut_along_their_keys(num_sms, cut, causal, dtype, out_dtype):
    """From one pair of CTAs that takes every tile in turn to many that share few."""
    check_prefill([130, 1, 300], [3000, 2000, 777], 3, causal, dtype, out_dtype, out_scale=0.5,
                  num_sms=num_sms, cut=cut)


def test_prefill_of_one_row_behind_many_keys():
    check_prefill([1], [20000], 1, num_sms=152, cut=True)


@pytest.mark.parametrize("scale", [0.0, 3.0])
def test_prefill_scales_of_cut_tiles(scale):
    check_prefill([100], [3000], 2, scale=scale, num_sms=16, cut=True)


def test_prefill_cut_tiles_given_a_workspace_captured_and_in_two_streams():
    lq, lk = [200, 40], [2500, 900]
    qo, ko = [0, 200, 240], [0, 2500, 3400]
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn((240, 2, 192), generator=g, device=DEV).to(BF)
    kv = torch.randn((3400, 2, 256), generator=g, device=DEV).to(BF)
    rope = torch.randn((3400, 64), generator=g, device=DEV).to(BF)
    k, v = kv[..., :128], kv[..., 128:]
    plan = api.batch_latent_prefill_plan(qo, ko, num_heads=2, return_lse=True, num_sms=24)
    assert plan.workspace_bytes > 0
    run = api.batch_latent_prefill_run
    with pytest.raises(L.PkaError) as e:
        run(plan, q, k, rope, v, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == L.PKA_ERR_WORKSPACE_TOO_SMALL
    out, lse = run(plan, q, k, rope, v)
    _, ref = ref_prefill(q, k, rope, v, qo, ko, 192 ** -0.5, True, 1.0, BF)
    assert_within(out, lse, ref)
    states = []
    for i in range(2):   # each stream has a workspace and outputs of its own
        states.append((torch.cuda.Stream(),
                       torch.full((plan.workspace_bytes // 4,), float("nan"), device=DEV),
                       torch.empty_like(out), torch.empty_like(lse)))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws, o, x in states:
            run(plan, q, k, rope, v, out=o, lse=x, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, _, o, x in states:
        assert torch.equal(o, out) and torch.equal(x, lse)
    s, ws, o, x = states[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(plan, q, k, rope, v, out=o, lse=x, workspace=ws)
    o.fill_(float("nan"))
    x.fill_(float("nan"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(x, lse)
    plan.check()


@pytest.mark.parametrize("out_dtype", [BF, FP])
def test_prefill_output_that_is_16_byte_aligned_only(out_dtype):
    g = torch.Generator(device=DEV).manual_seed(6)
    q, k, v = (torch.randn((150, 3, n), generator=g, device=DEV).to(BF) for n in (192, 128, 128))
    rope = torch.randn((150, 64), generator=g, device=DEV).to(BF)
    plan = api.batch_latent_prefill_plan([0, 150], [0, 150], num_heads=3, out_dtype=out_dtype)
    want = api.batch_latent_prefill_run(plan, q, k, rope, v)
    shift = 16 // want.element_size()
    room = torch.zeros(want.numel() + 2 * shift, dtype=out_dtype, device=DEV)
    out = room[shift:shift + want.numel()].view(want.shape)
    assert out.data_ptr() % 32 == 16
    api.batch_latent_prefill_run(plan, q, k, rope, v, out=out)
    assert torch.equal(out, want)
    assert bool((room[:shift] == 0).all()) and bool((room[-shift:] == 0).all())


def test_prefill_long():
    rows = set(random.Random(1).sample(range(3000 + 1500), 60)) | {0, 2999, 3000, 4499}
    check_prefill([3000, 1500], [3000, 4100], 5, rows=rows)


def test_prefill_ignores_what_lies_in_other_requests():
    """Keys and values of the next request, infinities and NaN included, are in the last
    tile of this one; they are masked, not multiplied by a zero weight."""
    g = torch.Generator(device=DEV).manual_seed(0)
    qo, ko = [0, 40], [0, 70]
    q = torch.randn((40, 2, 192), generator=g, device=DEV).to(BF)
    kv = torch.randn((140, 2, 256), generator=g, device=DEV).to(BF)
    rope = torch.randn((140, 64), generator=g, device=DEV).to(BF)
    kv[70:] = float("inf")
    kv[90:] = float("nan")
    rope[70:] = float("nan")
    qb = torch.cat([q, q])
    plan = api.batch_latent_prefill_plan([0, 40, 80], [0, 70, 140], num_heads=2, return_lse=True,
                                         causal=False)
    out, lse = api.batch_latent_prefill_run(plan, qb, kv[..., :128], rope, kv[..., 128:])
    plan.check()
    picked, ref = ref_prefill(q, kv[..., :128], rope, kv[..., 128:], qo, ko, 192 ** -0.5, False,
                              1.0, BF)
    assert_within(out[:40], lse[:40], ref)


def test_prefill_nan_in_a_key_reaches_the_rows_that_see_it():
    lq = lk = [70, 200]
    qo = [0, 70, 270]
    g = torch.Generator(device=DEV).manual_seed(3)
    q, kn, v, rope = (torch.randn(*s, generator=g, device=DEV).to(BF)
                      for s in ((270, 2, 192), (270, 2, 128), (270, 2, 128), (270, 64)))
    plan = api.batch_latent_prefill_plan(qo, qo, num_heads=2, causal=True, return_lse=True)
    good, good_lse = api.batch_latent_prefill_run(plan, q, kn, rope, v)
    kn[70 + 130] = float("nan")
    out, lse = api.batch_latent_prefill_run(plan, q, kn, rope, v)
    plan.check()
    assert torch.equal(out[:200], good[:200]) and torch.equal(lse[:200], good_lse[:200])
    assert bool(out[200:].isnan().all()) and bool(lse[200:].isnan().all())


def test_prefill_leaves_rows_behind_the_batch_and_can_be_captured():
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn((300, 3, 192), generator=g, device=DEV).to(BF)
    kv = torch.randn((400, 3, 256), generator=g, device=DEV).to(BF)
    rope = torch.randn((400, 64), generator=g, device=DEV).to(BF)
    qo, ko = [0, 5, 205], [0, 150, 350]
    plan = api.batch_latent_prefill_plan(qo, ko, num_heads=3, return_lse=True)
    out = torch.full((300, 3, 128), 7.0, dtype=BF, device=DEV)
    lse = torch.full((300, 3), 7.0, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.batch_latent_prefill_run(plan, q, kv[..., :128], rope, kv[..., 128:], out=out, lse=lse)
    for _ in range(2):
        q.mul_(0.5)
        graph.replay()
        plan.check()
        picked, ref = ref_prefill(q, kv[..., :128], rope, kv[..., 128:], qo, ko, 192 ** -0.5, True,
                                  1.0, BF)
        assert_within(out[picked], lse[picked], ref)
        assert bool((out[205:] == 7).all()) and bool((lse[205:] == 7).all())


def test_prefill_many_tiles_of_one_request():
    """Key runs long enough that every ring of the kernel turns many times, odd lengths."""
    rows = {0, 1, 255, 256, 300, 511, 512, 640}
    check_prefill([641], [5003], 2, rows=rows, causal=False)
    check_prefill([641, 2], [5003, 4097], 1, dtype=HF, rows=rows)


def test_prefill_refusals():
    plan = api.batch_latent_prefill_plan([0, 4], [0, 4], num_heads=2)
    q = torch.zeros((4, 2, 192), dtype=BF, device=DEV)
    k = torch.zeros((4, 2, 128), dtype=BF, device=DEV)
    r = torch.zeros((4, 64), dtype=BF, device=DEV)
    run = api.batch_latent_prefill_run
    with pytest.raises(ValueError, match="same strides"):
        run(plan, q, k, r, torch.zeros((4, 2, 256), dtype=BF, device=DEV)[..., :128])
    with pytest.raises(ValueError, match="q must be"):
        run(plan, q[:3], k, r, k)
    with pytest.raises(ValueError, match="k_rope must be"):
        run(plan, q, k, r[:, :32], k)
    with pytest.raises(ValueError, match="cpu"):
        run(plan, q, k, r.cpu(), k)
    with pytest.raises(L.PkaError, match="batch_latent_prefill_plan"):
        api.batch_prefill_run(plan, k, k, k)
    plain = api.batch_prefill_plan([0, 4], [0, 4], num_qo_heads=2, num_kv_heads=2)
    with pytest.raises(ValueError, match="batch_latent_prefill_plan"):
        run(plain, q, k, r, k)


# ---- together ----------------------------------------------------------------------

def test_serving_steps_from_an_empty_cache_captured_and_replayed():
    """Prompts into an empty cache and eight decode steps: pages and slots from the
    lengths, rows into the pool, absorbed decode over live lengths; the step is captured
    once and replayed.  Request 3 stays idle throughout."""
    B, H, dl, ps, D, width = 4, 20, 256, 16, 320, 8
    prompt = [37, 1, 64, 0]
    g = torch.Generator(device=DEV).manual_seed(5)
    pool = 40
    free = torch.randperm(pool, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(DEV)
    pages = torch.full((pool, ps, D), float("nan"), dtype=BF, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    history = [[] for _ in range(B)]

    rows = torch.randn((sum(prompt) + 6, D), generator=g, device=DEV).to(BF)
    t = api.paged_kv_tables(i32([0] * B), i32(prompt), free, i32([0]), table, page_size=ps,
                            num_slots=rows.shape[0], status=status)
    api.paged_latent_append(rows[:, :dl], rows[:, dl:], t.slot_map, pages, status=status)
    at = 0
    for b, n in enumerate(prompt):
        history[b] += list(rows[at:at + n])
        at += n

    lens, head = t.seq_lens.clone(), t.free_head.clone()
    new = i32([1, 1, 1, 0])
    x = torch.zeros((B, D), dtype=BF, device=DEV)
    q = torch.zeros((B, H, D), dtype=BF, device=DEV)
    plan = api.paged_latent_decode_plan([width * ps] * B, num_heads=H, page_size=ps, scale=0.06,
                                        max_pages_per_seq=width, num_pages=pool, latent_dim=dl,
                                        return_lse=True, freeze_seq_lens=False)
    out = torch.empty((B, H, dl), dtype=BF, device=DEV)
    lse = torch.empty((B, H), device=DEV)
    ws = torch.empty(max(1, plan.workspace_bytes), dtype=torch.uint8, device=DEV)

    def step():
        s = api.paged_kv_tables(lens, new, free, head, table, page_size=ps, num_slots=B,
                                status=status)
        api.paged_latent_append(x[:, :dl], x[:, dl:], s.slot_map, pages, status=status)
        api.paged_latent_decode_run(plan, q, pages, table, seq_lens_kv=s.seq_lens, out=out,
                                    lse=lse, workspace=ws)
        lens.copy_(s.seq_lens)
        head.copy_(s.free_head)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for k in range(8):
        x.copy_(torch.randn((B, D), generator=g, device=DEV))
        q.copy_(torch.randn((B, H, D), generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        api.check_status(status)
        plan.check()
        for i, b in enumerate([0, 1, 2]):
            history[b].append(x[i].clone())
        kv = [len(h) for h in history]
        assert lens.tolist() == kv
        dense = torch.full((B, width * ps, D), 0.0, dtype=BF, device=DEV)
        for b in range(B):
            if kv[b]:
                dense[b, :kv[b]] = torch.stack(history[b])
        ref = ref_decode(q, dense.view(-1, ps, D), torch.arange(B * width, device=DEV).view(B, -1),
                         kv, list(range(B + 1)), dl, 0.06, False, 1.0, BF)
        assert_within(out, lse, ref)
    used = [p for r in table.tolist() for p in r if p >= 0]
    assert len(used) == len(set(used)) == int(head)


def test_absorbed_decode_agrees_with_expanded_prefill():
    """One attention in its two forms: the last row of a prompt through the expanded
    prefill, and through the absorbed decode with its value projection behind it."""
    H, dl, n, ps = 6, 256, 150, 16
    g = torch.Generator(device=DEV).manual_seed(9)
    wk = torch.randn((H, 128, dl), generator=g, device=DEV, dtype=torch.float64) / 16
    wv = torch.randn((H, 128, dl), generator=g, device=DEV, dtype=torch.float64) / 16
    rows = torch.randn((n, dl + 64), generator=g, device=DEV).to(HF)
    c = rows[:, :dl].double()
    k = torch.einsum("nd,hed->nhe", c, wk).to(HF)
    v = torch.einsum("nd,hed->nhe", c, wv).to(HF)
    q = torch.randn((n, H, 192), generator=g, device=DEV).to(HF)
    plan = api.batch_latent_prefill_plan([0, n], [0, n], num_heads=H, return_lse=True, dtype=HF)
    out, lse = api.batch_latent_prefill_run(plan, q, k, rows[:, dl:], v)
    pages = torch.zeros((12, ps, dl + 64), dtype=HF, device=DEV)
    api.paged_latent_append(rows[:, :dl], rows[:, dl:], torch.arange(n, device=DEV), pages)
    qa = torch.cat([torch.einsum("the,hed->thd", q[-1:, :, :128].double(), wk).to(HF),
                    q[-1:, :, 128:]], -1)
    dplan = api.paged_latent_decode_plan([n], num_heads=H, page_size=ps, max_pages_per_seq=12,
                                         num_pages=12, scale=192 ** -0.5, latent_dim=dl,
                                         return_lse=True, dtype=HF, out_dtype=FP)
    oa, la = api.paged_latent_decode_run(dplan, qa, pages, torch.arange(12, device=DEV,
                                                                        dtype=torch.int32)[None])
    got = torch.einsum("thd,hed->the", oa.double(), wv)
    # q, k and v were rounded to half on the expanded side, the absorbed q on the other:
    # scores of up to ~200 terms of size ~1 each differ by a few 2^-11 after the scale
    assert float((la[0] - lse[-1]).abs().max()) < 0.02
    assert float((got[0] - out[-1].double()).abs().max()) < 0.02


# ---- kernels that run longer than any one of their waits may (2 s) -------------------

def took(run):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    r = run()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / 1e3, r


def test_prefill_of_one_pair_that_runs_for_seconds():
    """384 tiles of 2^20 keys on one pair of CTAs: every wait is for one tile at most."""
    lq, lk = 384 * 256, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(0)
    q, k, v, rope = (torch.randn(s, generator=g, device=DEV).to(BF) for s in
                     ((lq, 1, 192), (lk, 1, 128), (lk, 1, 128), (lk, 64)))
    plan = api.batch_latent_prefill_plan([0, lq], [0, lk], num_heads=1, causal=False, num_sms=1)
    seconds, out = took(lambda: api.batch_latent_prefill_run(plan, q, k, rope, v))
    plan.check()
    assert seconds > 2 and bool(out.isfinite().all())


@pytest.mark.parametrize("heads", [16, 128])
def test_decode_of_one_segment_that_runs_for_seconds(heads):
    """Requests that all see the same pages, one behind the other on one CTA (pair)."""
    batch, kv = 400, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(0)
    pages = torch.randn((64, 256, 320), generator=g, device=DEV).to(BF)
    table = torch.arange(64, dtype=torch.int32, device=DEV).repeat(batch, kv // (64 * 256))
    q = torch.randn((1, heads, 320), generator=g, device=DEV).to(BF).repeat(batch, 1, 1)
    plan = api.paged_latent_decode_plan([kv] * batch, num_heads=heads, page_size=256, scale=0.05,
                                        max_pages_per_seq=kv // 256, num_pages=64, latent_dim=256,
                                        num_sms=1, return_lse=True)
    seconds, (out, lse) = took(lambda: api.paged_latent_decode_run(plan, q, pages, table))
    plan.check()
    assert seconds > 2
    assert bool(out.isfinite().all()) and bool((out == out[0]).all()) and bool((lse == lse[0]).all())
