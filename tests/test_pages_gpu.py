"""Fork, release, compaction and page copies against plain Python, and their refusals."""

import random

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api
from tests import pages_ref as ref

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return dev([0])


def code_of(st):
    try:
        api.check_status(st)
    except L.PkaError as e:
        return e.code
    return L.PKA_OK


def pool_state(seed, batch, width, ps, kv_hi, family=1, spare=20, stride=None):
    """Lists (kv, tables, free, head, num_pages): families share half of the pages they all
    fill, page ids scattered, the list's head somewhere inside it with garbage before it."""
    r = random.Random(seed)
    kv = [r.randint(0, kv_hi) for _ in range(batch)]
    need = [-(-n // ps) for n in kv]
    total = sum(need) + spare
    ids = list(range(total + 7))
    r.shuffle(ids)   # 7 pages are in neither the tables nor the list
    tables, at = [], 0
    for b in range(batch):
        row = [-5] * width
        lead = b // family * family
        same = min(kv[x] // ps for x in range(lead, min(batch, lead + family))) // 2 if b != lead else 0
        row[:same] = tables[lead][:same] if same else []
        for j in range(same, need[b]):
            row[j] = ids[at]
            at += 1
        tables.append(row)
    head = at
    return kv, tables, [-9] * head + ids[at:total], head, len(ids)


def strided(tables, extra):
    """The tables on the device, in rows with `extra` further entries behind them."""
    t = torch.full((len(tables), len(tables[0]) + extra), -77, dtype=torch.int32, device="cuda")
    t[:, : len(tables[0])] = dev(tables)
    return t, t[:, : len(tables[0])]


SHAPES = [   # batch, width, page size, longest, family, extra row entries
    (2, 1, 16, 16, 1, 0),
    (3, 4, 1, 4, 2, 3),
    (17, 9, 16, 144, 3, 0),
    (40, 300, 48, 14000, 5, 5),
    (700, 33, 7, 230, 4, 1),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", [0, 1])
def test_fork(shape, seed):
    batch, width, ps, kv_hi, family, extra = shape
    kv, tables, free, head, _ = pool_state(seed, batch, width, ps, kv_hi, family, spare=batch + 3)
    r = random.Random(seed)
    rows = r.sample(range(batch), batch)
    cut = r.randint(1, batch - 1)
    children = rows[cut:]
    parents = [r.choice(rows[:cut]) for _ in children]
    whole, t = strided(tables, extra)
    st = status()
    got = api.paged_kv_fork(dev(parents), dev(children), dev(kv), dev(free), dev([head]), t, page_size=ps, status=st)
    api.check_status(st)
    want = ref.fork(parents, children, kv, free, head, tables, ps)
    assert t.tolist() == want[0]
    assert got.seq_lens.tolist() == want[1]
    assert got.src_pages.tolist() == want[2] and got.dst_pages.tolist() == want[3]
    assert got.free_head.tolist() == [want[4]]
    if extra:
        assert bool((whole[:, width:] == -77).all())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("part", [0.0, 0.3, 1.0])
def test_free(shape, part):
    batch, width, ps, kv_hi, family, extra = shape
    kv, tables, free, head, pages = pool_state(3, batch, width, ps, kv_hi, family)
    rows = random.Random(5).sample(range(batch), int(batch * part))
    whole, t = strided(tables, extra)
    f, st = dev(free), status()
    got = api.paged_kv_free(dev(rows), dev(kv), f, dev([head]), t, page_size=ps, num_pages=pages, status=st)
    api.check_status(st)
    want = ref.release(rows, kv, free, head, tables, ps)
    assert f.tolist() == want[0]
    assert got.seq_lens.tolist() == want[1] and got.free_head.tolist() == [want[2]]
    assert t.tolist() == tables


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("spare", [0, 1, 50, 4000])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(shape, spare, in_place):
    batch, width, ps, kv_hi, family, extra = shape
    kv, tables, free, head, pages = pool_state(7, batch, width, ps, kv_hi, family, spare=spare)
    whole, t = strided(tables, extra)
    f, st = dev(free), status()
    out = dict(block_tables_out=t, free_pages_out=f) if in_place else {}
    got = api.paged_kv_compact(dev(kv), f, dev([head]), t, page_size=ps, num_pages=pages, status=st, **out)
    api.check_status(st)
    want = ref.compact(kv, free, head, tables, ps)
    n = len(want[2])
    assert got.num_moves.tolist() == [n]
    assert got.src_pages.tolist() == want[2] + [-1] * (got.src_pages.numel() - n)
    assert got.dst_pages.tolist() == want[3] + [-1] * (got.dst_pages.numel() - n)
    assert got.block_tables.tolist() == want[0]
    assert got.free_pages.tolist() == want[1]
    if in_place:
        assert got.block_tables is t and got.free_pages is f
        if extra:
            assert bool((whole[:, width:] == -77).all())
    else:
        assert t.tolist() == tables and f.tolist() == free


def test_compact_of_many_pages_and_a_bound_on_moves():
    """More pages than one word a thread; exactly as many moves as there is room for, and one
    fewer, which is refused."""
    kv, tables, free, head, pages = pool_state(11, 64, 1100, 3, 3300, 1, spare=300000)
    want = ref.compact(kv, free, head, tables, 3)
    n = len(want[2])
    assert n > 1000
    args = (dev(kv), dev(free), dev([head]), dev(tables))
    got = api.paged_kv_compact(*args, page_size=3, num_pages=pages, src_pages=dev([0] * n), dst_pages=dev([0] * n))
    assert got.src_pages.tolist() == want[2] and got.dst_pages.tolist() == want[3]
    assert got.block_tables.tolist() == want[0] and got.free_pages.tolist() == want[1]
    st = status()
    got = api.paged_kv_compact(*args, page_size=3, num_pages=pages, src_pages=dev([0] * (n - 1)),
                               dst_pages=dev([0] * (n - 1)), status=st)
    assert code_of(st) == L.PKA_ERR_DEVICE_CAPACITY
    assert got.num_moves.tolist() == [0] and set(got.src_pages.tolist()) == {-1}
    assert got.block_tables.tolist() == tables and got.free_pages.tolist() == free


def test_largest_pool():
    """2^22 pages: release and compaction of the highest ones."""
    pages, ps = 1 << 22, 16
    tables = [[pages - 1, pages - 3, -1], [pages - 1, 5, 0]]
    kv = [2 * ps, 3 * ps]
    free = [-1] * 4 + [1, 2, 3, pages - 2]
    f = dev(free)
    got = api.paged_kv_free(dev([0]), dev(kv), f, dev([4]), dev(tables), page_size=ps, num_pages=pages)
    assert f.tolist() == [-1] * 3 + [pages - 3] + free[4:] and got.free_head.tolist() == [3]
    got = api.paged_kv_compact(dev(kv), dev(free), dev([4]), dev(tables), page_size=ps, num_pages=pages)
    want = ref.compact(kv, free, 4, tables, ps)
    assert got.block_tables.tolist() == want[0] and got.free_pages.tolist() == want[1]


def _fork_refused(parents, children, kv, free, head, tables, ps, code):
    st, t = status(), dev(tables)
    got = api.paged_kv_fork(dev(parents), dev(children), dev(kv), dev(free), dev([head]), t, page_size=ps, status=st)
    assert code_of(st) == code
    assert t.tolist() == tables and got.seq_lens.tolist() == kv and got.free_head.tolist() == [head]
    assert set(got.src_pages.tolist()) == {-1} and set(got.dst_pages.tolist()) == {-1}


def test_fork_refusals_change_nothing():
    kv, tables, ps = [20, 16, 0, 5], [[0, 1], [2, 7], [8, 9], [3, 6]], 16
    free = [4, 5]
    bounds, capacity = L.PKA_ERR_DEVICE_BOUNDS, L.PKA_ERR_DEVICE_CAPACITY
    for parents, children in (([0, 0], [2, 2]), ([0], [0]), ([0, 1], [1, 2]), ([4], [2]), ([0], [-1]), ([-1], [2]),
                              ([0], [4])):
        _fork_refused(parents, children, kv, free, 0, tables, ps, bounds)
    _fork_refused([0, 0], [1, 2], kv, free, 1, tables, ps, capacity)      # two tails, one page
    _fork_refused([0], [2], kv, free, -1, tables, ps, capacity)
    _fork_refused([1], [2], kv, free, 3, tables, ps, capacity)            # a head past the list
    _fork_refused([0], [2], [33, 16, 0, 5], free, 0, tables, ps, capacity)
    _fork_refused([0], [2], [-1, 16, 0, 5], free, 0, tables, ps, capacity)


def test_fork_of_full_pages_needs_no_free_page():
    t, st = dev([[3, 4], [0, 0]]), status()
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    got = api.paged_kv_fork(dev([0]), dev([1]), dev([32, 0]), empty, dev([0]), t, page_size=16, status=st)
    api.check_status(st)
    assert t.tolist() == [[3, 4], [3, 4]] and got.seq_lens.tolist() == [32, 32]
    assert got.src_pages.tolist() == [-1] and got.dst_pages.tolist() == [-1]
    got = api.paged_kv_fork(empty, empty, dev([32, 0]), empty, dev([0]), t, page_size=16)
    assert got.seq_lens.tolist() == [32, 0] and got.src_pages.numel() == 0


def test_release_refusals_change_nothing():
    kv, tables, free, pages = [20, 16], [[0, 1], [2, 3]], [7, 7, 5], 8

    def refused(rows, code, kv=kv, head=2, tables=tables):
        st, f, t = status(), dev(free), dev(tables)
        got = api.paged_kv_free(dev(rows), dev(kv), f, dev([head]), t, page_size=16, num_pages=pages, status=st)
        assert code_of(st) == code
        assert f.tolist() == free and got.seq_lens.tolist() == kv and got.free_head.tolist() == [head]

    refused([0, 0], L.PKA_ERR_DEVICE_BOUNDS)
    refused([2], L.PKA_ERR_DEVICE_BOUNDS)
    refused([-1], L.PKA_ERR_DEVICE_BOUNDS)
    refused([0], L.PKA_ERR_DEVICE_CAPACITY, head=1)
    refused([0], L.PKA_ERR_DEVICE_CAPACITY, head=4)
    refused([0], L.PKA_ERR_DEVICE_CAPACITY, head=-1)
    refused([0], L.PKA_ERR_DEVICE_CAPACITY, kv=[33, 16])
    refused([0], L.PKA_ERR_DEVICE_CAPACITY, kv=[20, -1])
    refused([0], L.PKA_ERR_DEVICE_BOUNDS, tables=[[0, 1], [8, 3]])
    refused([0], L.PKA_ERR_DEVICE_BOUNDS, tables=[[0, -1], [2, 3]])


def test_compact_refusals_change_nothing():
    kv, tables, free, pages = [20, 16], [[0, 5], [2, 3]], [-1, 4, 6], 8

    def refused(code, kv=kv, head=1, tables=tables, free=free):
        st = status()
        got = api.paged_kv_compact(dev(kv), dev(free), dev([head]), dev(tables), page_size=16, num_pages=pages, status=st)
        assert code_of(st) == code
        assert got.block_tables.tolist() == tables and got.free_pages.tolist() == free
        assert got.num_moves.tolist() == [0] and set(got.src_pages.tolist()) == {-1}

    refused(L.PKA_ERR_DEVICE_BOUNDS, free=[-1, 5, 6])         # in use and free
    refused(L.PKA_ERR_DEVICE_BOUNDS, free=[-1, 4, 4])         # listed twice
    refused(L.PKA_ERR_DEVICE_BOUNDS, free=[-1, 4, 8])
    refused(L.PKA_ERR_DEVICE_BOUNDS, head=0)                  # -1 is no page
    refused(L.PKA_ERR_DEVICE_BOUNDS, tables=[[0, 8], [2, 3]])
    refused(L.PKA_ERR_DEVICE_CAPACITY, kv=[20, 33])
    refused(L.PKA_ERR_DEVICE_CAPACITY, head=4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
@pytest.mark.parametrize("page", [(1, 16, 1), (3, 5, 16), (8, 64, 128), (7, 33, 16)])
def test_copy(dtype, page):
    g = torch.Generator(device="cuda").manual_seed(1)
    n = 40
    a = torch.randint(0, 200, (n, *page), generator=g, device="cuda").to(dtype)
    wide = torch.randint(0, 200, (n, 2, *page), generator=g, device="cuda").to(dtype)
    b = wide[:, 1]   # one half of a combined pool
    order = torch.randperm(n, generator=torch.Generator().manual_seed(2)).tolist()
    src, dst = order[:15], order[15:30]
    src[3], dst[7] = -1, -2
    ra, rw = a.clone(), wide.clone()
    for s, d in zip(src, dst):
        if s >= 0 and d >= 0:
            ra[d], rw[d, 1] = ra[s], rw[s, 1]
    st = status()
    api.paged_kv_copy([a, b], dev(src), dev(dst), status=st)
    api.check_status(st)
    assert torch.equal(a, ra) and torch.equal(wide, rw)


@pytest.mark.parametrize("count", [-3, 0, 2, 5, 9])
def test_copy_counts_and_reports(count):
    pools = [torch.arange(12 * 16, device="cuda", dtype=torch.float32).view(12, 16) * (i + 1) for i in range(70)]
    before = [p.clone() for p in pools]
    src, dst = [0, 1, 2, 12, 4], [6, 7, 8, 9, 13]
    st = status()
    api.paged_kv_copy(api.KvPools(pools), dev(src), dev(dst), count=dev([count]), status=st)
    n = max(0, min(5, count))
    assert code_of(st) == (L.PKA_ERR_DEVICE_BOUNDS if n > 3 else L.PKA_OK)
    for p, q in zip(pools, before):
        for s, d in list(zip(src, dst))[:min(n, 3)]:
            q[d] = q[s]
        assert torch.equal(p, q)


def test_offsets_past_32_bits():
    """Pages whose byte offsets in the pool pass 2^32, and entries whose bits lie far apart."""
    pool = torch.zeros((70000, 65536), dtype=torch.uint8, device="cuda")
    pool[69999] = 3
    pool[65540, ::2] = 9
    api.paged_kv_copy([pool], dev([69999, 65540]), dev([1, 69000]))
    assert bool((pool[1] == 3).all()) and bool((pool[69000, ::2] == 9).all()) and int(pool[69000].sum()) == 9 * 32768


def test_captured_and_replayed():
    """A fork with its copies, and the release of what it made, in one graph: each replay gives
    the same tables, and the free list's pages come back."""
    kv, tables, free, head, pages = pool_state(9, 12, 8, 16, 120, 1, spare=12)
    kv[10] = kv[11] = 0
    parents, children = [1, 2], [10, 11]
    kv[1], kv[2] = kv[1] | 1, kv[2] | 1   # both with a last page that is not full
    need = [-(-n // 16) for n in kv]
    pool = torch.arange(pages, device="cuda", dtype=torch.float32)[:, None].repeat(1, 16)
    t, f, h, lens, st = dev(tables), dev(free), dev([head]), dev(kv), status()
    p, c = dev(parents), dev(children)
    pools = api.KvPools([pool])

    def step():
        a = api.paged_kv_fork(p, c, lens, f, h, t, page_size=16, status=st)
        api.paged_kv_copy(pools, a.src_pages, a.dst_pages, status=st)
        b = api.paged_kv_free(c, a.seq_lens, f, a.free_head, t, page_size=16, num_pages=pages, status=st)
        return a, b

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = step()
    for _ in range(3):
        pool.copy_(torch.arange(pages, device="cuda", dtype=torch.float32)[:, None].expand(-1, 16))
        graph.replay()
        api.check_status(st)
        assert b.free_head.tolist() == [head] and b.seq_lens.tolist() == kv
        for q, r in zip(parents, children):
            full = kv[q] // 16
            assert t[r, :full].tolist() == tables[q][:full]
            assert pool[t[r, full].item(), 0].item() == tables[q][full]
    assert sorted(f.tolist()[head:]) == sorted(free[head:])


def test_streams():
    """Calls on a given stream come behind that stream's work and allocate from it."""
    kv, tables, free, head, pages = pool_state(13, 9, 6, 16, 96, 2, spare=16)
    side = torch.cuda.Stream()
    t, f = torch.zeros((9, 6), dtype=torch.int32, device="cuda"), torch.zeros(len(free), dtype=torch.int32, device="cuda")
    src_t, src_f, lens, h = dev(tables), dev(free), dev(kv), dev([head])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        t.copy_(src_t)
        f.copy_(src_f)
    got = api.paged_kv_compact(lens, f, h, t, page_size=16, num_pages=pages, stream=side)
    side.synchronize()
    want = ref.compact(kv, free, head, tables, 16)
    assert got.block_tables.tolist() == want[0] and got.free_pages.tolist() == want[1]


@pytest.mark.parametrize("pages", [1, 31, 32, 33, 700000, 1100000, 3000001])
def test_pools_of_several_ranges(pages):
    """Pools of one page, of a word and a bit more, and of more pages than a CTA marks at once,
    whose ids lie all over them."""
    r = random.Random(pages)
    batch, width, ps = 30, 80, 2
    ids = r.sample(range(pages), min(pages, 2400))
    kv, tables, at = [], [], 0
    for b in range(batch):
        n = min(r.randint(0, width), len(ids) - at)
        kv.append(n * ps)
        tables.append(ids[at:at + n] + [-2 ** 31] * (width - n))
        at += n
    spare = ids[at:]
    free = [-1] * at + spare
    rows = [b for b in range(batch) if b % 3 == 0]
    f, st = dev(free), status()
    got = api.paged_kv_free(dev(rows), dev(kv), f, dev([at]), dev(tables), page_size=ps, num_pages=pages, status=st)
    want = ref.release(rows, kv, free, at, tables, ps)
    assert f.tolist() == want[0] and got.seq_lens.tolist() == want[1] and got.free_head.tolist() == [want[2]]
    got = api.paged_kv_compact(dev(kv), dev(free), dev([at]), dev(tables), page_size=ps, num_pages=pages, status=st)
    api.check_status(st)
    new, lst, src, dst = ref.compact(kv, free, at, tables, ps)
    assert got.block_tables.tolist() == new and got.free_pages.tolist() == lst
    assert got.src_pages.tolist()[:len(src)] == src and got.dst_pages.tolist()[:len(dst)] == dst
    if pages > 2400:   # the same free page twice, seen by different CTAs or by one
        for i, j in ((at, at + 1), (at, len(free) - 1)):
            twice = list(free)
            twice[i] = twice[j]
            got = api.paged_kv_compact(dev(kv), dev(twice), dev([at]), dev(tables), page_size=ps, num_pages=pages,
                                       status=st)
            assert code_of(st) == L.PKA_ERR_DEVICE_BOUNDS and got.block_tables.tolist() == tables
