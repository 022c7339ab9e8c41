"""The latent planner and the host-side checks of the latent entry points (no GPU)."""
import ctypes
import random

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api


def _plan(seq, **kw):
    args = dict(num_heads=16, page_size=16, max_pages_per_seq=20000, num_pages=100000, scale=0.05,
                num_sms=152, host_only=True)
    args.update(kw)
    return api.paged_latent_decode_plan(seq, **args)


def _tiles(n):
    return max(1, -(-n // 64))


@pytest.mark.parametrize("heads", [1, 16, 17, 64, 128, 1024])
@pytest.mark.parametrize("seed", range(6))
def test_pieces_cover_every_request_once(heads, seed):
    r = random.Random(seed)
    B = r.choice([1, 2, 7, 64, 300])
    top = r.choice([1, 100, 9000, 200000])
    seq = [r.randint(0, top) for _ in range(B)]
    qo = [0]
    for _ in range(B):
        qo.append(qo[-1] + r.choice([0, 1, 1, 1, 3]))
    plan = _plan(seq, num_heads=heads, qo_indptr=qo)
    items, segs = plan.export()
    inf = plan.info
    rows = max(b - a for a, b in zip(qo, qo[1:])) * heads
    assert inf["row_tile"] == (16 if rows <= 16 else 32 if rows <= 32 else 64 if rows <= 64 else 128)
    assert inf["row_blocks"] == max(1, -(-rows // inf["row_tile"]))
    ctas = inf["row_blocks"] * (2 if inf["row_tile"] == 128 else 1)
    assert inf["num_segments"] <= max(1, 152 // ctas)
    assert segs[0] == 0 and segs[-1] == len(items) and all(a < b for a, b in zip(segs, segs[1:]))
    at, parts = {}, {}
    for b, lo, hi, part in items:
        assert lo == at.get(b, 0) < hi
        at[b] = hi
        parts.setdefault(b, []).append(part)
    partial = 0
    for b, n in enumerate(seq):
        if qo[b + 1] == qo[b]:
            assert b not in at
            continue
        assert at[b] == _tiles(n)
        assert parts[b] == ([-1] if len(parts[b]) == 1 else list(range(len(parts[b]))))
        if len(parts[b]) > 1:
            partial += len(parts[b]) * (qo[b + 1] - qo[b]) * heads
    assert inf["partial_rows"] == partial
    assert inf["num_split"] == sum(len(p) > 1 for p in parts.values())
    assert inf["workspace_bytes"] >= partial * (512 + 1) * 4


def test_segments_carry_equal_loads():
    r = random.Random(3)
    seq = [r.randint(512, 8192) for _ in range(64)]
    items, segs = _plan(seq).export()
    loads = [sum(hi - lo for _, lo, hi, _ in items[a:b]) for a, b in zip(segs, segs[1:])]
    mean = sum(_tiles(n) for n in seq) / 152
    assert max(loads) <= 1.15 * mean + 6


@pytest.mark.parametrize("kw,code", [
    (dict(latent_dim=128), L.PKA_ERR_UNSUPPORTED),
    (dict(rope_dim=32), L.PKA_ERR_UNSUPPORTED),
    (dict(num_heads=1025), L.PKA_ERR_UNSUPPORTED),
    (dict(num_heads=0), L.PKA_ERR_INVALID_ARG),
    (dict(page_size=12), L.PKA_ERR_UNSUPPORTED),
    (dict(page_size=264), L.PKA_ERR_UNSUPPORTED),
    (dict(page_size=0), L.PKA_ERR_UNSUPPORTED),
    (dict(seq=[-1, 3]), L.PKA_ERR_INVALID_ARG),
    (dict(seq=[330, 3], max_pages_per_seq=20), L.PKA_ERR_INVALID_ARG),
    (dict(q_len=0), L.PKA_ERR_INVALID_ARG),
    (dict(qo_indptr=[0, 3, 2]), L.PKA_ERR_INVALID_ARG),
    (dict(qo_indptr=[1, 3, 4]), L.PKA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), L.PKA_ERR_INVALID_ARG),
    (dict(output_scale=float("inf")), L.PKA_ERR_INVALID_ARG),
    (dict(num_pages=0), L.PKA_ERR_INVALID_ARG),
    (dict(num_pages=2 ** 31 - 1), L.PKA_ERR_INVALID_ARG),
    (dict(num_sms=2000), L.PKA_ERR_INVALID_ARG),
    (dict(num_heads=1024, q_len=65), L.PKA_ERR_UNSUPPORTED),
    (dict(q_len=2 ** 30, num_heads=1), L.PKA_ERR_INVALID_ARG),
])
def test_decode_plan_rejects(kw, code):
    kw = dict(kw)
    with pytest.raises(L.PkaError) as e:
        _plan(kw.pop("seq", [100, 50]), **kw)
    assert e.value.code == code


def test_decode_plan_rejects_offsets_of_another_batch():
    with pytest.raises(ValueError, match="qo_indptr"):
        _plan([100, 50], qo_indptr=[0, 1])
    plan = _plan([100, 50], qo_indptr=[0, 1, 2])
    with pytest.raises(ValueError, match="qo_indptr"):
        plan.update([100, 50, 3], qo_indptr=[0, 1, 2])


def test_update_replans_and_a_failed_one_changes_nothing():
    plan = _plan([100, 50])
    plan.update([7000, 3, 0])
    items, _ = plan.export()
    assert {b for b, *_ in items} == {0, 1, 2} and plan.total_q == 3
    with pytest.raises(L.PkaError):
        plan.update([-4])
    assert plan.export()[0] == items


def test_host_only_plan_does_not_run():
    plan = _plan([100])
    rc = L.lib().paged_latent_decode_run(plan.handle, None, 0, 0, None, 0, None, 0, None, None,
                                         None, None, 0, None)
    assert rc == L.PKA_ERR_INVALID_ARG and b"HOST_ONLY" in L.lib().pka_last_error()
    assert L.lib().paged_latent_decode_plan_check(plan.handle, None) == L.PKA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(nope_dim=64), L.PKA_ERR_UNSUPPORTED),
    (dict(rope_dim=0), L.PKA_ERR_UNSUPPORTED),
    (dict(value_dim=256), L.PKA_ERR_UNSUPPORTED),
    (dict(num_heads=0), L.PKA_ERR_INVALID_ARG),
    (dict(sm_scale=-1.0), L.PKA_ERR_UNSUPPORTED),
    (dict(kv=[0, 10, 20]), L.PKA_ERR_INVALID_ARG),      # fewer keys than causal rows
    (dict(qo=[0, 10, 5]), L.PKA_ERR_INVALID_ARG),
])
def test_prefill_plan_rejects(kw, code):
    kw = dict(kw)
    qo, kv = kw.pop("qo", [0, 10, 30]), kw.pop("kv", [0, 10, 30])
    args = dict(num_heads=2, host_only=True)
    args.update(kw)
    with pytest.raises(L.PkaError) as e:
        api.batch_latent_prefill_plan(qo, kv, **args)
    assert e.value.code == code


def test_prefill_plan_tiles():
    plan = api.batch_latent_prefill_plan([0, 300, 300, 310], [0, 300, 300, 400], num_heads=4,
                                         host_only=True)
    assert plan.num_tiles == (2 + 1) * 4        # 256 rows of one head each
    with pytest.raises(ValueError, match="same length"):
        api.batch_latent_prefill_plan([0, 3], [0, 3, 4], num_heads=1, host_only=True)


def _fake(n=256):
    """A 256-byte aligned host address: the entry points reject before using it."""
    buf = (ctypes.c_uint8 * (2 * n + 256))()
    return buf, (ctypes.addressof(buf) + 255) & ~255


def test_tables_entry_point_rejects():
    lib = L.lib()
    keep, p = _fake(4096)
    a = [p + 256 * i for i in range(12)]

    def call(batch=2, free_n=4, ps=16, stride=8, width=8, slots=4, kv=a[0], seq=a[5], status=a[9],
             slot_map=a[7]):
        return lib.paged_kv_tables(kv, a[1], batch, a[2], free_n, a[3], ps, a[4], stride, width, seq,
                                   a[6], slot_map, slots, a[8], status, None)

    for kw in (dict(batch=0), dict(free_n=-1), dict(ps=0), dict(ps=65537), dict(stride=7),
               dict(width=0, stride=0), dict(slots=0), dict(kv=None), dict(kv=a[0] + 2),
               dict(seq=a[0]), dict(seq=a[0] + 4), dict(slot_map=a[7] + 4), dict(seq=a[6] + 4)):
        assert call(**kw) == L.PKA_ERR_INVALID_ARG, kw


def test_append_entry_point_rejects():
    lib = L.lib()
    keep, p = _fake()

    def call(latent=p, ls=512, rope=p, rs=64, dl=512, dr=64, n=1, pages=p, num_pages=2, ps=16,
             sp=16 * 576, dtype=0):
        return lib.paged_latent_append(latent, ls, rope, rs, dl, dr, p, n, pages, num_pages, ps, sp,
                                       dtype, None, None)

    for kw in (dict(latent=None), dict(latent=p + 8), dict(ls=4), dict(ls=-8), dict(dl=4),
               dict(dr=12), dict(dr=0), dict(rope=None), dict(n=-1), dict(pages=p + 2),
               dict(num_pages=0), dict(ps=0), dict(sp=16 * 576 - 8), dict(sp=16 * 576 + 4)):
        assert call(**kw) == L.PKA_ERR_INVALID_ARG, kw
    assert call(dtype=L.PKA_DTYPE_F32) == L.PKA_ERR_UNSUPPORTED


def test_binding_wants_cuda_tensors(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="current device"):
        api.check_status(z)
    with pytest.raises(ValueError, match="current device"):
        api.paged_latent_append(torch.zeros((1, 64), dtype=torch.bfloat16), None,
                                torch.zeros(1, dtype=torch.int64),
                                torch.zeros((1, 8, 64), dtype=torch.bfloat16))


@pytest.mark.parametrize("qo,kv,heads,num_sms,cut", [
    ([0, 300], [0, 300], 4, 152, False),          # short tiles stay whole
    ([0, 256], [0, 64 * 1000], 1, 1, False),      # one pair takes everything in turn
    ([0, 256], [0, 64 * 1000], 1, 152, True),     # one tile, shared out
    ([0, 256], [0, 64 * 1000], 152, 152, False),  # as many equal tiles as pairs
    ([0, 256], [0, 64 * 1000], 200, 152, True),   # a second round a third full
    ([0, 0], [0, 5], 3, 152, False),              # no rows
])
def test_prefill_plan_cuts_tiles_only_where_pairs_end_unevenly(qo, kv, heads, num_sms, cut):
    plan = api.batch_latent_prefill_plan(qo, kv, num_heads=heads, causal=False, num_sms=num_sms,
                                         host_only=True)
    assert (plan.workspace_bytes > 0) == cut
    assert plan.workspace_bytes % (256 * 129 * 4) == 0      # whole states: 256 rows and their LSEs
    assert plan.workspace_bytes // (256 * 129 * 4) <= plan.num_tiles + num_sms


@pytest.mark.parametrize("num_sms", [-1, 5000])
def test_prefill_plan_refuses_sm_counts(num_sms):
    with pytest.raises(L.PkaError) as e:
        api.batch_latent_prefill_plan([0, 3], [0, 3], num_heads=1, num_sms=num_sms, host_only=True)
    assert e.value.code == L.PKA_ERR_INVALID_ARG
