"""Decode behind shared prefixes against 64-bit attention over every request's own table."""

import ctypes
import math
import random

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api
from tests import prefix_ref as ref

pytestmark = pytest.mark.gpu

D = 128


def make(groups, *, heads, kv_heads, ps, q_lens=None, dtype=torch.bfloat16, seed=0, spare_cols=0, scale=None,
         live=None):
    """groups: [(prefix pages, [own keys of each request])]; q_lens per request."""
    r = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kv, indptr, pre = [], [0], []
    for pages, own in groups:
        pre.append(pages)
        indptr.append(indptr[-1] + len(own))
        kv += [pages * ps + n for n in own]
    need = [-(-n // ps) for n in kv]
    total = sum(need) + 5 + sum(pages for pages, own in groups if not own)
    ids = list(range(total))
    r.shuffle(ids)
    tables, at = [], 0
    width = max(need) + spare_cols
    for gi, (pages, own) in enumerate(groups):
        shared = ids[at:at + pages]
        at += pages
        for b in range(indptr[gi], indptr[gi + 1]):
            mine = ids[at:at + need[b] - pages]
            at += len(mine)
            tables.append(shared + mine + [-3] * (width - need[b]))
    qo = [0]
    for n in q_lens or [1] * len(kv):
        qo.append(qo[-1] + n)
    k, v = (torch.randn((total, kv_heads, ps, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((qo[-1], heads, D), generator=g, device="cuda").to(dtype)
    return dict(kv=kv, groups=indptr, pre=pre, tables=tables, qo=qo, q=q, k=k, v=v, ps=ps, heads=heads,
                kv_heads=kv_heads, dtype=dtype, scale=scale or 1 / math.sqrt(D), width=width)


def plan_of(c, **kw):
    a = dict(num_qo_heads=c["heads"], num_kv_heads=c["kv_heads"], page_size=c["ps"], max_pages_per_seq=c["width"],
             num_pages=c["k"].shape[0], qo_indptr=c["qo"], scale=c["scale"], return_lse=True, dtype=c["dtype"], min_shared_bytes=0)
    a.update(kw)
    return api.paged_prefix_decode_plan(c["kv"], c["groups"], c["pre"], **a)


def table(c):
    return torch.tensor(c["tables"], dtype=torch.int32, device="cuda")


def close(got, want, v, dtype, out_dtype):
    """The output is a mean of v with weights p rounded to the input type (half a step of each,
    so of the mean of |v|, at most the largest |v| of what is averaged) and one rounding to the
    output type; the 32-bit sums add 2^-18 of it, the LSE's difference of scores likewise."""
    out, lse = got
    eps = torch.finfo(dtype).eps / 2
    eps_out = torch.finfo(out_dtype).eps / 2
    top = float(v[v.isfinite()].abs().max())
    bound = eps_out * want[0].abs() + (eps + 2.0 ** -18) * top
    err = (out.double() - want[0]).abs()
    assert bool((err <= bound).all()), f"out off by {float(err.max())}, allowed {float(bound.max())}"
    if lse is not None:
        bound = 2.0 ** -18 * want[1].abs().clamp(min=1) + 2.0 ** -16
        assert bool(((lse.double() - want[1]).abs() <= bound).all())


def check(c, causal=False, out_dtype=None, sinks=None, bmm2_scale=1.0, plan=None, pieces=True, **kw):
    p = plan or plan_of(c, causal=causal, out_dtype=out_dtype, bmm2_scale=bmm2_scale)
    assert bool(p.info["shared"]) == pieces
    got = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], table(c), sinks=sinks, **kw)
    p.check()
    want = ref.decode(c["q"], c["k"], c["v"], c["tables"], c["kv"], c["qo"], causal=causal, scale=c["scale"],
                      sinks=sinks, bmm2_scale=bmm2_scale)
    close(got, want, c["v"] * bmm2_scale, c["dtype"], out_dtype or c["dtype"])
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ps", [16, 32, 48, 64, 96, 256])
def test_page_sizes(dtype, ps):
    n = -(-900 // ps)
    check(make([(n, [1, 17, 100, 64, 3])], heads=8, kv_heads=2, ps=ps, dtype=dtype))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 8), (5, 1), (14, 2), (32, 4), (64, 1), (300, 2)])
def test_head_groups(heads, kv_heads):
    check(make([(13, [5, 40, 16, 1, 77, 9, 130])], heads=heads, kv_heads=kv_heads, ps=16, seed=heads))


@pytest.mark.parametrize("pages", [1, 2, 3, 4, 5, 9, 60, 400])
def test_prefix_lengths(pages):
    """One page, pieces that end inside a tile of 64 keys, and many pieces."""
    check(make([(pages, [20] * 6 + [300])], heads=8, kv_heads=2, ps=16, seed=pages))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sms,dense", [(1, 1), (2, 1), (3, 0), (152, 0)])
def test_shapes_of_the_prefix_kernel(sms, dense, dtype):
    """Many tiles a CTA take two CTAs an SM, few one: the same batch on few SMs and on all."""
    c = make([(60, [1 + i % 8 for i in range(150)])], heads=8, kv_heads=2, ps=16, dtype=dtype)
    p = plan_of(c, num_sms=sms)
    assert p.info["dense"] == dense
    check(c, plan=p)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("kv_heads", [1, 2, 8])
def test_rows_of_many_states(kv_heads, sinks):
    """Few rows behind many keys: several warps join a row's states.  More rows: one does."""
    c = make([(512, [700, 1, 5000])], heads=8, kv_heads=kv_heads, ps=16, seed=kv_heads)
    check(c, sinks=torch.randn(8, device="cuda") if sinks else None)
    c = make([(512, [700, 1, 5000] + [20] * 57)], heads=8, kv_heads=kv_heads, ps=16, seed=kv_heads)
    check(c, sinks=torch.randn(8, device="cuda") if sinks else None)


@pytest.mark.parametrize("requests", [2, 63, 64, 65, 150])
def test_row_tiles(requests):
    """Rows that fill part of a CTA's 128, of a pair's 256, and several pairs."""
    check(make([(20, [1 + (7 * i) % 50 for i in range(requests)])], heads=8, kv_heads=2, ps=16))


@pytest.mark.parametrize("causal", [False, True])
def test_several_groups_and_packed_queries(causal):
    groups = [(10, [50, 30, 20]), (0, [40, 17]), (33, [12] * 9), (4, [100]), (2, [11, 12])]
    q_lens = [1, 3, 2, 4, 1, 1, 2, 3, 4, 5, 6, 7, 8, 9, 3, 11, 12]
    check(make(groups, heads=12, kv_heads=4, ps=16, q_lens=q_lens, dtype=torch.float16), causal=causal)


def test_requests_that_end_with_the_prefix():
    """No key of their own behind the shared pages; causal rows of which the first sees just them."""
    check(make([(6, [0, 0, 5, 0])], heads=8, kv_heads=2, ps=32))
    check(make([(6, [0, 0])], heads=8, kv_heads=2, ps=16))
    check(make([(8, [2, 2, 40])], heads=4, kv_heads=2, ps=16, q_lens=[3, 3, 3]), causal=True)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_output_types_sinks_and_scales(out_dtype):
    c = make([(30, [10, 200, 31])], heads=8, kv_heads=2, ps=16, seed=3)
    sinks = torch.randn(8, device="cuda") * 3
    check(c, out_dtype=out_dtype, sinks=sinks, bmm2_scale=0.5)
    c["scale"] = -0.2
    check(c, out_dtype=out_dtype)
    c["scale"] = 1e-30
    check(c, out_dtype=out_dtype)


def test_scale_zero():
    c = make([(5, [10, 3])], heads=4, kv_heads=2, ps=16)
    c["scale"] = 0.0
    check(c)


def test_large_scores():
    """Weights that one key takes almost alone, in the prefix for some rows, in their own keys for others."""
    c = make([(40, [60, 70, 5, 300])], heads=8, kv_heads=2, ps=16, seed=8)
    c["scale"] = 4.0
    check(c)


def test_strided_queries_and_combined_pools():
    c = make([(30, [10, 200, 31, 16])], heads=8, kv_heads=2, ps=16, seed=5)
    wide = torch.zeros((4, 3, 8, D), dtype=c["dtype"], device="cuda")
    wide[:, 1] = c["q"]
    both = torch.stack([c["k"], c["v"]], 1)   # [pages, 2, ...]
    c["q"], c["k"], c["v"] = wide[:, 1], both[:, 0], both[:, 1]
    check(c)
    heads_first = c["q"].transpose(0, 1).contiguous().transpose(0, 1)
    c["q"] = heads_first
    check(c)


def test_what_lies_past_the_keys_does_not_matter():
    """Infinities and NaN behind each request's keys and in the pool's other pages; table entries
    behind a request's pages."""
    c = make([(3, [10, 2, 31]), (2, [5, 6])], heads=8, kv_heads=2, ps=48, seed=6, spare_cols=3)
    used = set()
    for b, n in enumerate(c["kv"]):
        row = c["tables"][b][: -(-n // 48)]
        used |= set(row)
        if n % 48:
            for pool, bad in ((c["k"], float("nan")), (c["v"], float("inf"))):
                pool[row[-1], :, n % 48:] = bad
    for page in set(range(c["k"].shape[0])) - used:
        c["k"][page] = float("nan")
        c["v"][page] = float("nan")
    got = check(c)
    assert bool(got[0].isfinite().all())


def test_infinite_values_and_nan_in_the_prefix():
    c = make([(5, [10, 7])], heads=4, kv_heads=2, ps=16, seed=4)
    c["v"][c["tables"][0][1], 0, 3, 9] = float("inf")
    c["v"][c["tables"][0][2], 1, 5, 11] = float("nan")
    p = plan_of(c)
    out, lse = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], table(c))
    want, _ = ref.decode(c["q"], c["k"], c["v"], c["tables"], c["kv"], c["qo"], causal=False, scale=c["scale"])
    assert torch.equal(out.isinf(), want.isinf()) and torch.equal(out.isnan(), want.isnan())
    assert bool(out[:, :2, 9].isinf().all()) and bool(out[:, 2:, 11].isnan().all()) and bool(lse.isfinite().all())


def test_table_entries_outside_the_pool_read_as_zeros():
    c = make([(6, [20, 20])], heads=4, kv_heads=2, ps=16, seed=2)
    bad = [list(r) for r in c["tables"]]
    for r in bad:
        r[2], r[4] = -1, 2 ** 31 - 1
    p = plan_of(c)
    got = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], torch.tensor(bad, dtype=torch.int32, device="cuda"))
    p.check()
    for pool in (c["k"], c["v"]):
        pool[c["tables"][0][2]] = 0
        pool[c["tables"][0][4]] = 0
    want = ref.decode(c["q"], c["k"], c["v"], c["tables"], c["kv"], c["qo"], causal=False, scale=c["scale"])
    close(got, want, c["v"], c["dtype"], c["dtype"])


@pytest.mark.parametrize("shared", [False, True])
def test_check_tables(shared):
    """An entry outside the pool in any row, rows that do not begin alike; entries that no run reads."""
    c = make([(6, [20, 40, 1]), (0, [30]), (3, [0, 16])], heads=4, kv_heads=2, ps=16, seed=2, spare_cols=2)
    p = plan_of(c if shared else c | {"pre": [0, 0, 0]}, freeze_seq_lens=False)
    live = torch.tensor(c["kv"], dtype=torch.int32, device="cuda")
    p.check_tables(table(c), live)
    p.check()

    def fails(row, col, page, lens=live):
        t = table(c)
        t[row, col] = page
        p.check_tables(t, lens)
        try:
            p.check()
        except L.PkaError as e:
            assert e.code == L.PKA_ERR_DEVICE_BOUNDS
            p.check()   # read and cleared
            return True
        return False

    n = c["k"].shape[0]
    for row, col in ((0, 0), (0, 5), (1, 8), (2, 6), (3, 1), (4, 2), (5, 3)):
        assert fails(row, col, n) and fails(row, col, -1)
        assert not fails(row, col, c["tables"][row][col])
    assert not fails(1, 9, n) and not fails(4, 3, -1)        # behind the row's pages
    other = c["tables"][3][0]
    assert fails(1, 3, other) == shared and fails(5, 2, other) == shared
    assert not fails(1, 6, other)                            # a request's own page
    # a request that has become shorter: its own pages are not read, the shared ones are
    short = live.clone()
    short[1] = 97
    assert not fails(1, 8, n, short) and fails(1, 6, n, short)
    short[1] = 1
    assert fails(1, 5, n, short) == shared
    with pytest.raises(ValueError):
        p.check_tables(table(c)[:5], live)
    with pytest.raises(ValueError):
        p.check_tables(table(c), live[:4])
    with pytest.raises(ValueError):
        p.check_tables(table(c).long(), live)


def test_live_lengths():
    """Planned for the longest; each run reads the lengths as they are."""
    c = make([(20, [400, 300, 350]), (6, [100, 90])], heads=8, kv_heads=2, ps=16, seed=7)
    p = plan_of(c, freeze_seq_lens=False)
    for cut in ([0, 0, 0, 0, 0], [399, 1, 350, 100, 0], [100, 299, 17, 3, 89]):
        now = [n - x for n, x in zip(c["kv"], cut)]
        lens = torch.tensor(now, dtype=torch.int32, device="cuda")
        got = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], table(c), seq_lens_kv=lens)
        want = ref.decode(c["q"], c["k"], c["v"], c["tables"], now, c["qo"], causal=False, scale=c["scale"])
        close(got, want, c["v"], c["dtype"], c["dtype"])


def test_update_and_rows_behind_the_last():
    c = make([(20, [40, 30, 35])], heads=8, kv_heads=2, ps=16, seed=1)
    p = plan_of(c)
    check(c, plan=p)
    d = make([(7, [40, 30]), (50, [35, 900, 8])], heads=8, kv_heads=2, ps=16, seed=2)
    d["width"] = c["width"]
    # more pages than the plan's table holds are refused, and the plan stays as it was
    with pytest.raises(Exception):
        p.update(d["kv"], d["groups"], d["pre"], qo_indptr=d["qo"])
    check(c, plan=p)
    e = make([(4, [40, 30]), (12, [35, 90, 8])], heads=8, kv_heads=2, ps=16, seed=2, spare_cols=5)
    p = plan_of(e)
    f = make([(3, [20, 20, 20]), (9, [10, 10])], heads=8, kv_heads=2, ps=16, seed=3)
    f["tables"] = [r + [-1] * (e["width"] - len(r)) for r in f["tables"]]
    n = e["k"].shape[0]
    for pool in ("k", "v"):
        f[pool] = torch.cat([f[pool], f[pool].new_zeros((n, *f[pool].shape[1:]))])[:n]
    p.update(f["kv"], f["groups"], f["pre"], qo_indptr=f["qo"])
    out = torch.full((f["qo"][-1] + 4, 8, D), 7.0, dtype=c["dtype"], device="cuda")
    lse = torch.full((f["qo"][-1] + 4, 8), 7.0, device="cuda")
    f["q"] = torch.cat([f["q"], f["q"][:2]])
    got = api.paged_prefix_decode_run(p, f["q"], f["k"], f["v"], table(f), out=out, lse=lse)
    T = f["qo"][-1]
    want = ref.decode(f["q"][:T], f["k"], f["v"], f["tables"], f["kv"], f["qo"], causal=False, scale=f["scale"])
    close((got[0][:T], got[1][:T]), want, f["v"], f["dtype"], f["dtype"])
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())


def test_update_between_shared_and_not():
    """A plan that comes to share nothing, and again something: each time as a plan of its own."""
    c = make([(30, [40, 30, 300]), (5, [9, 9])], heads=8, kv_heads=2, ps=16, seed=1)
    p = plan_of(c)
    for _ in range(2):
        check(c, plan=p)
        p.update(c["kv"], c["groups"], [0, 0], qo_indptr=c["qo"])
        check(c, plan=p, pieces=False)
        p.update(c["kv"], c["groups"], c["pre"], qo_indptr=c["qo"])
    p.update(c["kv"], [0, 0, 5], [0, 0], qo_indptr=c["qo"])
    p.update(c["kv"], [0, 2, 5], [30, 0], qo_indptr=c["qo"])
    check(c, plan=p)
    none = plan_of(c | {"pre": [0, 0]})
    none.update(c["kv"], c["groups"], c["pre"], qo_indptr=c["qo"])
    check(c, plan=none)


@pytest.mark.parametrize("shared", [False, True])
def test_update_that_fails_keeps_the_plan(shared):
    """An update that needs more memory while a stream of this thread captures is refused by CUDA: the
    plan runs as before, shared or not, and later updates work."""
    cudart = ctypes.CDLL("libcudart.so.13")
    c = make([(30, [40, 30, 300]), (5, [9, 9])], heads=8, kv_heads=2, ps=16, seed=1)
    p = plan_of(c if shared else c | {"pre": [0, 0]})
    check(c, plan=p, pieces=shared)
    info, ws = p.info, p.workspace_bytes
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), ctypes.c_void_p()
    n = 4096
    assert cudart.cudaStreamBeginCapture(ctypes.c_void_p(s.cuda_stream), 1) == 0
    try:
        with pytest.raises(L.PkaError):
            p.update([480] * n, [0, n], [30], stream=s)
    finally:
        cudart.cudaStreamEndCapture(ctypes.c_void_p(s.cuda_stream), ctypes.byref(graph))
        cudart.cudaGetLastError()
    assert p.info == info and p.workspace_bytes == ws
    check(c, plan=p, pieces=shared)
    p.update(c["kv"], c["groups"], c["pre"], qo_indptr=c["qo"])
    check(c, plan=p)


def test_captured_and_replayed():
    c = make([(50, [40, 30, 35, 1])], heads=16, kv_heads=2, ps=16, seed=1)
    p = plan_of(c, freeze_seq_lens=False)
    t, lens = table(c), torch.tensor(c["kv"], dtype=torch.int32, device="cuda")
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], t, seq_lens_kv=lens, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], t, seq_lens_kv=lens, workspace=ws)
    for cut in (0, 1, 30):
        now = [max(n - cut, 800) for n in c["kv"]]
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        c["q"].normal_()
        ws.fill_(255)   # nothing in the workspace is kept from one run to the next
        graph.replay()
        want = ref.decode(c["q"], c["k"], c["v"], c["tables"], now, c["qo"], causal=False, scale=c["scale"])
        close(got, want, c["v"], c["dtype"], c["dtype"])


def test_the_same_answer_every_time_and_on_another_stream():
    c = make([(200, [40, 300, 35, 1] * 8)], heads=32, kv_heads=8, ps=16, seed=1)
    p = plan_of(c)
    first = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], table(c))
    for _ in range(5):
        again = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], table(c))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    side = torch.cuda.Stream()
    t = table(c)
    side.wait_stream(torch.cuda.current_stream())
    again = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], t, stream=side)
    side.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
