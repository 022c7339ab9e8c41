"""One batch through the page pool's operators as a server would run them: prompts appended with
their rotation, requests forked, decoded behind the prefix that they share, grown apart, released
and compacted.  What every request holds is kept beside the pools, and each layer's attention
is compared with the 64-bit one over that."""

import math

import pytest
import torch

from paged_kv_attention_32_gb300 import api
from tests import pages_ref
from tests.test_prefix_gpu import close
from tests.test_rope_append_gpu import close as close_rows

pytestmark = pytest.mark.gpu

D, HQ, HKV, LAYERS = 128, 8, 2, 2


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    def __init__(self, rows, ps, pages, dtype, seed):
        self.ps, self.pages, self.dtype, self.width = ps, pages, dtype, 40
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.tables = torch.full((rows, self.width), -1, dtype=torch.int32, device="cuda")
        self.kv = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.free, self.head = ints(order), ints([0])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        # unwritten pages hold NaN: nothing may read them
        self.k = [torch.full((pages, HKV, ps, D), math.nan, dtype=dtype, device="cuda") for _ in range(LAYERS)]
        self.v = [torch.full((pages, HKV, ps, D), math.nan, dtype=dtype, device="cuda") for _ in range(LAYERS)]
        self.pools = api.KvPools(self.k + self.v)
        self.held = [[] for _ in range(rows)]   # per row: per token a list of (k, v) by layer
        self.inv_freq = 1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)

    def append(self, new):
        """new[b] tokens more for each row; returns the step's rotated queries by layer."""
        total = sum(new)
        at = torch.cat([torch.arange(n, n + m) for n, m in zip(self.kv.tolist(), new)]).to(torch.int32).cuda()
        t = api.paged_kv_tables(self.kv, ints(new), self.free, self.head, self.tables, page_size=self.ps,
                                num_slots=total + 3, status=self.status)
        self.kv, self.head = t.seq_lens, t.free_head
        slots = t.slot_map[:total]
        qs, rows = [], []
        for k_pages, v_pages in zip(self.k, self.v):
            x = torch.randn((total + 3, HQ + 2 * HKV, D), generator=self.g, device="cuda").to(self.dtype)
            q, k, v = x.split([HQ, HKV, HKV], dim=1)
            q_out = api.paged_rope_append(k, v, t.slot_map, k_pages, v_pages, q=q,
                                          positions=torch.cat([at, ints([0] * 3)]), inv_freq=self.inv_freq,
                                          status=self.status)
            got = [p.transpose(1, 2).reshape(-1, HKV, D)[slots] for p in (k_pages, v_pages)]
            close_rows(got[0], pages_ref.rotate(k[:total], at[None], self.inv_freq, [D // 2], "halves"), self.dtype)
            close_rows(q_out[:total], pages_ref.rotate(q[:total], at[None], self.inv_freq, [D // 2], "halves"), self.dtype)
            assert torch.equal(got[1], v[:total])
            qs.append(q_out[:total].contiguous())
            rows.append(got)
        i = 0
        for b, n in enumerate(new):
            for _ in range(n):
                self.held[b].append([(k[i], v[i]) for k, v in rows])
                i += 1
        api.check_status(self.status)
        assert self.kv.tolist() == [len(h) for h in self.held]
        return qs

    def attend(self, rows, qs, plan, run):
        """Each layer's attention of one query per row against what the rows hold."""
        for layer, q in enumerate(qs):
            out, lse = run(plan, q, self.k[layer], self.v[layer], self.tables[rows].contiguous())
            want, want_lse = torch.zeros(out.shape, dtype=torch.float64, device="cuda"), torch.zeros(lse.shape, dtype=torch.float64, device="cuda")
            for i, b in enumerate(rows):
                k, v = (torch.stack([t[layer][j] for t in self.held[b]], 1).double() for j in (0, 1))
                k, v = (x.repeat_interleave(HQ // HKV, 0) for x in (k, v))
                x = torch.einsum("hd,hnd->hn", q[i].double(), k) / math.sqrt(D)
                want[i] = torch.einsum("hn,hnd->hd", torch.softmax(x, 1), v)
                want_lse[i] = torch.logsumexp(x, 1) / math.log(2)
            close((out, lse), (want, want_lse), torch.stack([t[layer][1] for b in rows for t in self.held[b]]), self.dtype, self.dtype)

    def plans(self, rows, group, prefix):
        kw = dict(num_qo_heads=HQ, num_kv_heads=HKV, page_size=self.ps, max_pages_per_seq=self.width,
                  num_pages=self.pages, return_lse=True, dtype=self.dtype)
        lens = [len(self.held[b]) for b in rows]
        return (api.paged_decode_plan(lens, **kw),
                api.paged_prefix_decode_plan(lens, group, prefix, min_shared_bytes=0, **kw))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ps", [16, 48])
def test_a_batch_from_prompts_to_compaction(ps, dtype):
    b = Batch(8, ps, 160, dtype, ps)
    b.append([5 * ps + 7, 0, 0, 0, 3 * ps, 0, 1, 0])          # prompts; a page ends in row 4
    # rows 1 to 3 continue row 0, row 5 row 4
    f = api.paged_kv_fork(ints([0, 0, 0, 4]), ints([1, 2, 3, 5]), b.kv, b.free, b.head, b.tables,
                          page_size=ps, status=b.status)
    b.kv, b.head = f.seq_lens, f.free_head
    api.paged_kv_copy(b.pools, f.src_pages, f.dst_pages, status=b.status)
    for parent, child in ((0, 1), (0, 2), (0, 3), (4, 5)):
        b.held[child] = list(b.held[parent])
    tables = b.tables.tolist()
    assert all(tables[r][:5] == tables[0][:5] and tables[r][5] != tables[0][5] for r in (1, 2, 3))

    rows = [0, 1, 2, 3, 4, 5, 6]
    for step in range(2):                                      # all grow apart
        q = b.append([1, 1, 1 + ps * step, 1, 1, 1, 1, 0])
        last = [0, 1, 2 + ps * step, 3 + ps * step, 4 + ps * step, 5 + ps * step, 6 + ps * step]
        q = [x[last].contiguous() for x in q]
        plain, prefix = b.plans(rows, [0, 4, 6, 7], [5, 3, 0])
        assert prefix.info["shared"] == 1
        b.attend(rows, q, plain, api.paged_decode_run)
        b.attend(rows, q, prefix, api.paged_prefix_decode_run)

    # rows 0 and 4 end; what they share lives on in the others
    r = api.paged_kv_free(ints([0, 4]), b.kv, b.free, b.head, b.tables, page_size=ps, num_pages=b.pages, status=b.status)
    b.kv, b.head = r.seq_lens, r.free_head
    b.held[0], b.held[4] = [], []
    rows = [1, 2, 3, 5, 6]
    q = [x[[0, 1, 2, 3, 4]].contiguous() for x in b.append([0, 1, 1, 1, 0, 1, 1, 0])]
    plain, prefix = b.plans(rows, [0, 3, 4, 5], [5, 3, 0])
    b.attend(rows, q, plain, api.paged_decode_run)
    b.attend(rows, q, prefix, api.paged_prefix_decode_run)

    c = api.paged_kv_compact(b.kv, b.free, b.head, b.tables, page_size=ps, num_pages=b.pages, status=b.status)
    api.paged_kv_copy(b.pools, c.src_pages, c.dst_pages, count=c.num_moves, status=b.status)
    b.tables, b.free = c.block_tables, c.free_pages
    used = {p for t, n in zip(b.tables.tolist(), b.kv.tolist()) for p in t[: -(-n // ps)]}
    assert used == set(range(len(used)))
    b.attend(rows, q, plain, api.paged_decode_run)
    b.attend(rows, q, prefix, api.paged_prefix_decode_run)

    # the freed rows serve new prompts out of the compacted pool
    q = b.append([2 * ps, 1, 1, 1, 9, 1, 1, 4])
    rows = [0, 1, 2, 3, 4, 5, 6, 7]
    ends = [2 * ps - 1, 2 * ps, 2 * ps + 1, 2 * ps + 2, 2 * ps + 11, 2 * ps + 12, 2 * ps + 13, 2 * ps + 17]
    q = [x[ends].contiguous() for x in q]
    plain, prefix = b.plans(rows, [0, 1, 4, 8], [0, 5, 0])
    b.attend(rows, q, plain, api.paged_decode_run)
    b.attend(rows, q, prefix, api.paged_prefix_decode_run)
    api.check_status(b.status)


def test_two_streams_and_two_pools_at_once():
    """Two batches of their own on two streams, each with its plan and pools: neither disturbs
    the other, at the same time and in turn."""
    batches = [Batch(5, 16, 80, torch.bfloat16, s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in batches]
    work = []
    for b in batches:
        b.append([100, 0, 0, 0, 33])
        f = api.paged_kv_fork(ints([0, 0, 0]), ints([1, 2, 3]), b.kv, b.free, b.head, b.tables, page_size=16, status=b.status)
        b.kv, b.head = f.seq_lens, f.free_head
        api.paged_kv_copy(b.pools, f.src_pages, f.dst_pages, status=b.status)
        for r in (1, 2, 3):
            b.held[r] = list(b.held[0])
        q = b.append([1] * 5)
        _, prefix = b.plans(range(5), [0, 4, 5], [6, 0])
        work.append((q, prefix))
    want = [[api.paged_prefix_decode_run(p, q[i], b.k[i], b.v[i], b.tables) for i in range(LAYERS)]
            for b, (q, p) in zip(batches, work)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for n, (b, (q, p), s) in enumerate(zip(batches, work, streams)):
            got[n].append([api.paged_prefix_decode_run(p, q[i], b.k[i], b.v[i], b.tables, stream=s) for i in range(LAYERS)])
    torch.cuda.synchronize()
    for n in range(2):
        for outs in got[n]:
            for (out, lse), (w, wl) in zip(outs, want[n]):
                assert torch.equal(out, w) and torch.equal(lse, wl)
        work[n][1].check()
