"""The page pool's operators at the ends of their ranges, against the same plain lists."""

import random

import pytest
import torch

from paged_kv_attention_32_gb300 import api
from tests import pages_ref as ref
from tests.test_pages_gpu import code_of, dev, pool_state, status

pytestmark = pytest.mark.gpu


def free_and_compare(kv, tables, free, head, rows, ps, pages):
    f, st = dev(free), status()
    got = api.paged_kv_free(dev(rows), dev(kv), f, dev([head]), dev(tables), page_size=ps, num_pages=pages, status=st)
    api.check_status(st)
    want = ref.release(rows, kv, free, head, tables, ps)
    assert torch.equal(f, dev(want[0])) and torch.equal(got.seq_lens, dev(want[1])) and got.free_head.tolist() == [want[2]]


def compact_and_compare(kv, tables, free, head, ps, pages):
    st = status()
    got = api.paged_kv_compact(dev(kv), dev(free), dev([head]), dev(tables), page_size=ps, num_pages=pages, status=st)
    api.check_status(st)
    want = ref.compact(kv, free, head, tables, ps)
    n = len(want[2])
    assert got.num_moves.tolist() == [n]
    assert got.src_pages[:n].tolist() == want[2] and got.dst_pages[:n].tolist() == want[3]
    assert torch.equal(got.block_tables, dev(want[0])) and torch.equal(got.free_pages, dev(want[1]))


@pytest.mark.parametrize("batch,width,kv_hi", [(300, 300, 4799), (97, 1029, 16464), (2048, 40, 639)])
def test_large_tables(batch, width, kv_hi):
    """More entries than one CTA takes: rows of one piece, of three that end inside, and many rows."""
    kv, tables, free, head, pages = pool_state(batch, batch, width, 16, kv_hi, 4, spare=500)
    r = random.Random(batch)
    for part in (1, batch // 3, batch):
        free_and_compare(kv, tables, free, head, r.sample(range(batch), part), 16, pages)
    compact_and_compare(kv, tables, free, head, 16, pages)


def test_pages_all_over_the_largest_pool():
    """Entries in every range that the marks of 2^22 pages take, rows of many lengths."""
    pages, ps, r = 1 << 22, 16, random.Random(1)
    kv = [r.choice([0, 1, 16, 300, 5000, 8192]) for _ in range(200)]
    need = [-(-n // ps) for n in kv]
    ids = r.sample(range(pages), sum(need) + 5000)
    tables, at = [], 0
    for n in need:
        tables.append(ids[at:at + n] + [pages + 3] * (512 - n))
        at += n
    tables[7][:1], kv[7], need[7] = [0], 16, 1
    tables[8][:1], kv[8], need[8] = [pages - 1], 16, 1
    used = {p for t, n in zip(tables, need) for p in t[:n]}
    free = [-1] * 20000 + sorted(set(ids) - used, key=lambda p: p * 2654435761 % pages)
    free_and_compare(kv, tables, free, 20000, list(range(0, 200, 2)), ps, pages)
    compact_and_compare(kv, tables, free, 20000, ps, pages)


def test_as_many_rows_as_there_may_be():
    """16384 rows: one forked to all others, all but it released, what is left compacted."""
    B, ps = 16384, 16
    kv = [3 * ps + 5] + [0] * (B - 1)
    tables = [[70, 4, 30000, 9, -1]] + [[-1] * 5 for _ in range(B - 1)]
    free = [p for p in range(20000) if p not in (70, 4, 9)]
    t, f, st = dev(tables), dev(free), status()
    children = list(range(1, B))
    random.Random(2).shuffle(children)
    got = api.paged_kv_fork(dev([0] * (B - 1)), dev(children), dev(kv), f, dev([0]), t, page_size=ps, status=st)
    api.check_status(st)
    want = ref.fork([0] * (B - 1), children, kv, free, 0, tables, ps)
    assert torch.equal(t, dev(want[0])) and torch.equal(got.seq_lens, dev(want[1])) and got.free_head.tolist() == [want[4]]
    assert torch.equal(got.src_pages, dev(want[2])) and torch.equal(got.dst_pages, dev(want[3]))
    free_and_compare(want[1], want[0], free, want[4], children, ps, 30001)
    compact_and_compare(want[1], want[0], free, want[4], ps, 30001)


def test_nothing_to_do():
    """No forks, no rows, no free pages, no pages in use: outputs repeat inputs."""
    none = dev([])
    kv, tables = [0, 0, 33], [[7, 8, 9], [1, 1, 1], [5, 0, 2]]
    t, st = dev(tables), status()
    got = api.paged_kv_fork(none, none, dev(kv), none, dev([0]), t, page_size=16, status=st)
    assert got.seq_lens.tolist() == kv and got.free_head.tolist() == [0] and got.src_pages.numel() == 0
    got = api.paged_kv_free(none, dev(kv), none, dev([0]), t, page_size=16, num_pages=10, status=st)
    assert got.seq_lens.tolist() == kv and got.free_head.tolist() == [0]
    got = api.paged_kv_free(dev([0, 1]), dev(kv), none, dev([0]), t, page_size=16, num_pages=10, status=st)
    assert got.seq_lens.tolist() == kv and got.free_head.tolist() == [0]
    got = api.paged_kv_compact(dev(kv), none, dev([0]), t, page_size=16, num_pages=10, status=st)
    assert got.block_tables.tolist() == tables and got.num_moves.tolist() == [0]
    api.paged_kv_copy([torch.zeros((10, 8), device="cuda")], none, none, status=st)
    got = api.paged_kv_compact(dev([0] * 3), dev([4, 6]), dev([2]), t, page_size=16, num_pages=10, status=st)
    assert got.block_tables.tolist() == tables and got.free_pages.tolist() == [4, 6]
    api.check_status(st)
    # a release without room below the head is refused, and changes nothing
    f = dev([3])
    got = api.paged_kv_free(dev([2]), dev(kv), f, dev([0]), t, page_size=16, num_pages=10, status=st)
    assert code_of(st) != 0 and got.seq_lens.tolist() == kv and f.tolist() == [3] and got.free_head.tolist() == [0]


@pytest.mark.parametrize("ps", [1, 65536])
def test_smallest_and_largest_pages(ps):
    """Pages of one token are always full: forks take none.  Of 65536: lengths near 2^31."""
    width = 3 if ps == 1 else 32767
    full = width * ps
    kv, tables = [full, full - 1, 0], [[(7 * b + j) % 200003 for j in range(width)] for b in (0, 40000, 0)]
    t, st = dev(tables), status()
    used = {p for b, n in enumerate(kv) for p in tables[b][: -(-n // ps)]}
    free = [p for p in range(200003) if p not in used][:100]
    got = api.paged_kv_fork(dev([1]), dev([2]), dev(kv), dev(free), dev([0]), t, page_size=ps, status=st)
    api.check_status(st)
    want = ref.fork([1], [2], kv, free, 0, tables, ps)
    assert torch.equal(t, dev(want[0])) and got.seq_lens.tolist() == want[1]
    assert got.dst_pages.tolist() == want[3] and got.free_head.tolist() == [want[4]]
    compact_and_compare(want[1], want[0], free, want[4], ps, 200003)
    free = [-1] * 70000 + free[want[4]:]
    free_and_compare(want[1], want[0], free, 70000, [0], ps, 200003)


def test_odd_alignment():
    """Arrays that begin anywhere among 4 bytes, tables with rows of odd stride."""
    kv, tables, free, head, pages = pool_state(5, 40, 37, 16, 590, 4, spare=50)

    def off(x):
        whole = torch.full((len(x) + 3,), -77, dtype=torch.int32, device="cuda")
        whole[1: 1 + len(x)] = dev(x)
        return whole[1: 1 + len(x)]

    t = torch.full((40, 41), -77, dtype=torch.int32, device="cuda")[:, 1:38]
    t.copy_(dev(tables))
    f, st = off(free), status()
    got = api.paged_kv_free(off([3, 9, 4]), off(kv), f, off([head]), t, page_size=16, num_pages=pages, status=st,
                            seq_lens=off([0] * 40), free_head_out=off([0]))
    want = ref.release([3, 9, 4], kv, free, head, tables, 16)
    assert f.tolist() == want[0] and got.seq_lens.tolist() == want[1] and got.free_head.tolist() == [want[2]]
    w = ref.compact(want[1], want[0], want[2], tables, 16)
    for room in (60, len(w[2]), len(w[2]) + 5):   # the first too few
        g = api.paged_kv_compact(got.seq_lens, f, got.free_head, t, page_size=16, num_pages=pages, status=st,
                                 block_tables_out=t, src_pages=off([0] * room), dst_pages=off([0] * room),
                                 num_moves=off([0]))
        if room < len(w[2]):
            assert code_of(st) != 0 and t.tolist() == tables and g.free_pages.tolist() == want[0]
            continue
        api.check_status(st)
        assert t.tolist() == w[0] and g.free_pages.tolist() == w[1]
        assert g.src_pages.tolist() == w[2] + [-1] * (room - len(w[2])) and g.num_moves.tolist() == [len(w[2])]
        t.copy_(dev(tables))
