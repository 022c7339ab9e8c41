"""Cases of a shared K/V page pool at work: rotated keys and their values written to it,
requests forked over its pages, released and compacted, and decode attention for a batch
whose requests begin with the same pages, which are read once for all of them.

``run`` computes each operator either in elementary torch operations (32-bit, rounded
once; angles in 64) or, with ``own``, through the package's entry points.
"""

import math

import torch

own = False

D = 128   # head size of the paged K/V pools
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decode step of 64 requests: each one's new key, value and query rotated
        dict(name="rope_step_t64", op="rope", tokens=64, pad=0, heads=32, kv_heads=8, rotary=128,
             axes=1, pairs="halves", page=16, base=500000.0, far=131072, dtype="bf16"),
        # a chunk of a video prompt: three position axes, the chunk's tail padded
        dict(name="rope_video_t16384", op="rope", tokens=16200, pad=184, heads=32, kv_heads=8,
             rotary=128, axes=3, pairs="halves", page=64, base=1000000.0, far=30000, dtype="bf16"),
        # four sampled continuations of one prompt
        dict(name="fork_n4", op="fork", batch=16, forks=4, parents=1, kv_lo=500, kv_hi=1500, page=16,
             kv_heads=8, dtype="bf16"),
        # seven further beams for each of 64 prompts
        dict(name="fork_n448", op="fork", batch=512, forks=448, parents=64, kv_lo=100, kv_hi=4095,
             page=16, kv_heads=8, dtype="bf16"),
        # a few requests of a serving batch end
        dict(name="free_b64", op="free", batch=64, rows=5, family=4, kv_lo=100, kv_hi=4095, page=16),
        # a large batch of sampled families, half of which ends
        dict(name="free_b2048", op="free", batch=2048, rows=1024, family=8, kv_lo=100, kv_hi=8191,
             page=16),
        # a small pool after some requests have ended
        dict(name="compact_b16", op="compact", batch=16, family=2, kv_lo=100, kv_hi=1000, page=16,
             used=0.6, kv_heads=2, dtype="bf16"),
        # a large pool, a third of it free and spread over all of it
        dict(name="compact_b256", op="compact", batch=256, family=4, kv_lo=1000, kv_hi=8191, page=32,
             used=0.66, kv_heads=4, dtype="bf16"),
        # a few short continuations of a short prompt, bound by latency
        dict(name="prefix_b4", op="prefix", batch=4, groups=1, heads=8, kv_heads=2, page=16,
             prefix=256, suf_lo=1, suf_hi=64, q_len=1, causal=False, dtype="bf16"),
        # a serving batch behind one system prompt
        dict(name="prefix_b64_p8192", op="prefix", batch=64, groups=1, heads=32, kv_heads=8, page=16,
             prefix=8192, suf_lo=64, suf_hi=1024, q_len=1, causal=False, dtype="bf16"),
        # sampled families: four prompts, 32 continuations each
        dict(name="prefix_g4_b128", op="prefix", batch=128, groups=4, heads=32, kv_heads=8, page=32,
             prefix=16384, suf_lo=16, suf_hi=2048, q_len=1, causal=False, dtype="bf16"),
        # one long document under many questions, four drafted tokens a request to verify
        dict(name="prefix_spec_p65536", op="prefix", batch=32, groups=1, heads=64, kv_heads=8, page=64,
             prefix=65536, suf_lo=100, suf_hi=1000, q_len=4, causal=True, dtype="f16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "fork", "free", "compact", "prefix", "prefix", "prefix"])
    page = rng.choice([16, 16, 32, 48, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "rope":
        kv_heads = rng.choice([1, 2, 5, 8])
        heads = kv_heads * rng.choice([1, 3, 4, 8])
        tokens = _log(rng, 1, 16000 * 48 // max(48, heads + 2 * kv_heads))
        return dict(op=op, tokens=tokens, pad=rng.choice([0, 0, 1 + tokens // 9]), heads=heads,
                    kv_heads=kv_heads, rotary=rng.choice([128, 128, 64, 96, 32]),
                    axes=rng.choice([1, 1, 2, 3]), pairs=rng.choice(["halves", "halves", "neighbours"]),
                    page=page, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    far=_log(rng, 100, 500000), dtype=dtype)
    if op == "fork":
        batch = _log(rng, 2, 512)
        parents = _log(rng, 1, max(1, batch // 2))
        kv_hi = _log(rng, 1, 4095)
        return dict(op=op, batch=batch, forks=_log(rng, 1, batch - parents), parents=parents,
                    kv_lo=rng.choice([0, 1, kv_hi // 2]), kv_hi=kv_hi, page=page,
                    kv_heads=rng.choice([1, 2, 4]), dtype=dtype)
    if op == "free":
        batch, kv_hi = _log(rng, 1, 2048), _log(rng, 1, 8191)
        return dict(op=op, batch=batch, rows=_log(rng, 1, batch), family=rng.choice([1, 2, 4, 7]),
                    kv_lo=rng.choice([0, 1, kv_hi // 2]), kv_hi=kv_hi, page=page)
    if op == "compact":
        batch, kv_hi = _log(rng, 1, 256), _log(rng, 1, 4095)
        return dict(op=op, batch=batch, family=rng.choice([1, 2, 5]),
                    kv_lo=rng.choice([0, 1, kv_hi // 2]), kv_hi=kv_hi, page=page,
                    used=rng.choice([0.3, 0.6, 0.9, 1.0]), kv_heads=rng.choice([1, 2, 4]),
                    dtype=dtype)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    q_len = rng.choice([1, 1, 1, 2, 3])
    batch = _log(rng, 1, 96)
    prefix = _log(rng, page, 16384)
    suf_hi = _log(rng, q_len, 1500)
    return dict(op=op, batch=batch, groups=max(1, min(batch, rng.choice([1, 1, 2, 3, 5]))), heads=heads,
                kv_heads=kv_heads, page=page, prefix=prefix // page * page,
                suf_lo=rng.choice([q_len, max(q_len, suf_hi // 2)]), suf_hi=suf_hi, q_len=q_len,
                causal=q_len > 1 or rng.random() < 0.3, dtype=dtype)


# ---- inputs -------------------------------------------------------------------

def _gens(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    d = torch.Generator(device="cuda")
    d.manual_seed(seed + 1)
    return g, d


def _lens(case, g, n, lo="kv_lo", hi="kv_hi"):
    """The case's own ``n`` lengths, in an order of ``g``'s."""
    fixed = torch.Generator()
    fixed.manual_seed(0)
    x = torch.randint(case[lo], case[hi] + 1, (n,), generator=fixed, dtype=torch.int64)
    return x[torch.randperm(n, generator=g)]


def _sections(half, axes):
    """Frequencies per position axis: the first axis has the fewest."""
    return {1: (half,), 2: (half // 2, half - half // 2),
            3: (half // 4, half * 3 // 8, half - half // 4 - half * 3 // 8)}[axes]


def _pool(d, pages, case):
    return torch.randn((pages, case["kv_heads"], case["page"], D), generator=d, device="cuda",
                       dtype=_DTYPES[case["dtype"]])


def _int(x):
    return x.to(torch.int32).cuda()


def _family_tables(kv, ps, family, width):
    """Tables whose rows, ``family`` to a family, share the leading half of the pages
    that all of the family fill.  Returns (page number per entry or -1, pages in use)."""
    B = kv.numel()
    need = (kv + ps - 1) // ps
    head = torch.arange(B) // family * family
    fewest = torch.full((B,), 1 << 40, dtype=torch.int64).scatter_reduce(0, head, kv // ps, "amin")[head]
    shared = torch.where(head == torch.arange(B), 0, fewest // 2)
    count = need - shared
    first = count.cumsum(0) - count
    j = torch.arange(width)[None, :]
    own_page = first[:, None] + j - shared[:, None]
    table = torch.where(j < shared[:, None], own_page[head], own_page)
    return torch.where(j < need[:, None], table, -1), int(count.sum())


def _pool_pages(case, kv):
    """Pages of the pool: enough for the lengths ``kv`` even if no page were shared."""
    need = int(((kv + case["page"] - 1) // case["page"]).sum())
    return max(need + 1, int(need / case["used"])) if case["op"] == "compact" else need + 64


def prepare(case, seed):
    g, d = _gens(seed)
    s = dict(case)
    op = case["op"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "rope":
        T, n, ps = case["tokens"] + case["pad"], case["tokens"], case["page"]
        H, Hkv, half = case["heads"], case["kv_heads"], case["rotary"] // 2
        used = -(-n // ps)
        pages = used + 5
        order = torch.randperm(pages, generator=g, dtype=torch.int64)
        t = torch.arange(n, dtype=torch.int64)
        if n <= pages:   # a decode step: each token in a page of its own
            slots = order[t] * ps + torch.randint(0, ps, (n,), generator=g)
        else:
            slots = order[t // ps] * ps + t % ps
        slots = torch.cat([slots, torch.full((case["pad"],), -1, dtype=torch.int64)])
        t = torch.arange(T, dtype=torch.int64)
        if case["axes"] == 1 and n <= pages:
            pos = torch.randint(0, case["far"], (1, T), generator=g)
        else:   # frames of 24 x 40 patches behind some text
            grid = (t // 960, t // 40 % 24, t % 40) if case["axes"] == 3 else (t // 40, t % 40)
            grid = (t,) if case["axes"] == 1 else grid
            pos = torch.stack([x + int(torch.randint(0, case["far"], (1,), generator=g)) for x in grid])
        # one projection's output, as a model hands it on
        qkv = torch.randn((T, H + 2 * Hkv, D), generator=d, device="cuda", dtype=_DTYPES[case["dtype"]])
        freq = case["base"] ** (-torch.arange(half, dtype=torch.float64) / half)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:], slots=slots.cuda(),
                 pos=_int(pos), freq=freq.cuda(), sections=_sections(half, case["axes"]),
                 k_pages=_pool(d, pages, case), v_pages=_pool(d, pages, case), status=status)
    elif op == "fork":
        B, ps, n = case["batch"], case["page"], case["forks"]
        kv = torch.zeros(B, dtype=torch.int64)
        rows = torch.randperm(B, generator=g)
        parents, children = rows[:case["parents"]], rows[B - n:]
        kv[parents] = _lens(case, g, case["parents"])
        width = -(-max(case["kv_hi"], 1) // ps) + 1
        table, used = _family_tables(kv, ps, 1, width)
        pages = used + n + 9
        perm = torch.randperm(pages, generator=g, dtype=torch.int64)
        table = torch.where(table >= 0, perm[table.clamp(min=0)], -1)
        lead = int(torch.randint(0, 4, (1,), generator=g))
        s.update(parent=_int(parents[torch.arange(n) % case["parents"]]), child=_int(children),
                 kv_lens=_int(kv), table=_int(table), free=_int(torch.cat([torch.full((lead,), -1), perm[used:]])),
                 head=_int(torch.tensor([lead])), k_pages=_pool(d, pages, case),
                 v_pages=_pool(d, pages, case), status=status)
    elif op in ("free", "compact"):
        B, ps = case["batch"], case["page"]
        kv = _lens(case, g, B)
        width = -(-max(case["kv_hi"], 1) // ps) + 1
        table, used = _family_tables(kv, ps, case["family"], width)
        pages = _pool_pages(case, kv)
        perm = torch.randperm(pages, generator=g, dtype=torch.int64)
        table = torch.where(table >= 0, perm[table.clamp(min=0)], -1)
        # what a list that handed out these pages in turn looks like: its head behind them
        free = torch.cat([torch.full((used,), -1), perm[used:]])
        s.update(kv_lens=_int(kv), table=_int(table), free=_int(free), head=_int(torch.tensor([used])),
                 pages=pages, status=status)
        if op == "free":
            s["gone"] = _int(torch.randperm(B, generator=g)[:case["rows"]])
        else:
            s.update(k_pages=_pool(d, pages, case), v_pages=_pool(d, pages, case))
    else:
        B, ps, L, dt = case["batch"], case["page"], case["q_len"], _DTYPES[case["dtype"]]
        pre, group, suf = _prefix_lens(case, g)
        kv = pre[group] * ps + suf
        need = (kv + ps - 1) // ps
        width = int(need.max())
        j = torch.arange(width)[None, :]
        at = pre.cumsum(0) - pre                       # each group's first shared page
        tail = need - pre[group]
        first = int(pre.sum()) + tail.cumsum(0) - tail  # each request's first page of its own
        table = torch.where(j < pre[group][:, None], at[group][:, None] + j,
                            first[:, None] + j - pre[group][:, None])
        pages = int(pre.sum() + tail.sum()) + 3
        perm = torch.randperm(pages, generator=g, dtype=torch.int64)
        table = torch.where(j < need[:, None], perm[table.clamp(max=pages - 1)], -1)
        s.update(q=torch.randn((B * L, case["heads"], D), generator=d, device="cuda", dtype=dt),
                 k_pages=_pool(d, pages, case), v_pages=_pool(d, pages, case), table=_int(table),
                 kv_lens=_int(kv), kv_host=kv.tolist(), pre=pre.tolist(), scale=1.0 / math.sqrt(D),
                 ends=torch.bincount(group, minlength=case["groups"]).cumsum(0).tolist())
        if own:
            from paged_kv_attention_32_gb300 import api
            s["plan"] = api.paged_prefix_decode_plan(
                kv.to(torch.int32), [0] + s["ends"], s["pre"], num_qo_heads=case["heads"],
                num_kv_heads=case["kv_heads"], page_size=ps, max_pages_per_seq=width, num_pages=pages,
                q_len=L, causal=case["causal"], scale=s["scale"], return_lse=True, dtype=dt)
    if own and op in ("fork", "compact"):
        from paged_kv_attention_32_gb300 import api
        s["pools"] = api.KvPools([s["k_pages"], s["v_pages"]])
    return s


def _prefix_lens(case, g):
    """(shared pages of each group, group of each request, own keys of each request)."""
    B, n = case["batch"], case["groups"]
    pages = max(1, case["prefix"] // case["page"])
    pre = torch.tensor([max(1, pages * (i + 1) // n) for i in range(n)])
    return pre, torch.arange(B) * n // B, _lens(case, g, B, "suf_lo", "suf_hi")


# ---- one pass -------------------------------------------------------------------

def run(s):
    return _RUN[s["op"]](s)


def _angles(s):
    """Angles [tokens, rotary / 2] in 64 bits, each frequency with its axis' position."""
    axis = torch.repeat_interleave(torch.arange(s["axes"], device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"))
    return s["pos"].double()[axis].T * s["freq"]


def _turn(x, cos, sin, pairs):
    """The rotary part of ``x`` [tokens, heads, rotary] turned by the angles."""
    if pairs == "halves":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _rope(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        q = api.paged_rope_append(s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"], q=s["q"],
                                  positions=s["pos"], inv_freq=s["freq"], sections=s["sections"],
                                  pairs=s["pairs"], status=s["status"])
        return [q, s["k_pages"], s["v_pages"]]
    a, rd = _angles(s), s["rotary"]
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    q, k = (torch.cat([_turn(x[..., :rd].float(), cos, sin, s["pairs"]), x[..., rd:].float()], -1)
            .to(x.dtype) for x in (s["q"], s["k"]))
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    page, slot = slots // s["page"], slots % s["page"]
    s["k_pages"][page, :, slot] = k[keep]
    s["v_pages"][page, :, slot] = s["v"][keep]
    return [q, s["k_pages"], s["v_pages"]]


def _move(s, src, dst):
    keep = src >= 0
    src, dst = src[keep].long(), dst[keep].long()
    for pool in (s["k_pages"], s["v_pages"]):
        pool[dst] = pool[src]


def _fork(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        r = api.paged_kv_fork(s["parent"], s["child"], s["kv_lens"], s["free"], s["head"], s["table"],
                              page_size=s["page"], status=s["status"])
        api.paged_kv_copy(s["pools"], r.src_pages, r.dst_pages, status=s["status"])
        return [s["table"], r.seq_lens, r.src_pages, r.dst_pages, r.free_head, s["k_pages"], s["v_pages"]]
    ps, parent, child, table = s["page"], s["parent"].long(), s["child"].long(), s["table"]
    n = s["kv_lens"].long()[parent]
    full, part = n // ps, n % ps > 0
    rank = part.long().cumsum(0) - 1
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    tail = part[:, None] & (j == full[:, None])
    fresh = s["free"][(s["head"].long() + rank).clamp(0, s["free"].numel() - 1)]
    src = torch.where(part, table[parent, full.clamp(max=table.shape[1] - 1)], -1)
    dst = torch.where(part, fresh, -1)
    rows = torch.where(j < full[:, None], table[parent], table[child])
    table[child] = torch.where(tail, fresh[:, None], rows)
    lens = s["kv_lens"].clone()
    lens[child] = n.to(torch.int32)
    head = (s["head"] + part.sum()).to(torch.int32)
    _move(s, src, dst)
    return [table, lens, src, dst, head, s["k_pages"], s["v_pages"]]


def _marks(s, kv):
    """Which pages the first ceil(kv / page) entries of the rows hold."""
    need = (kv.long() + s["page"] - 1) // s["page"]
    inside = torch.arange(s["table"].shape[1], device="cuda")[None, :] < need[:, None]
    mark = torch.zeros(s["pages"] + 1, dtype=torch.bool, device="cuda")
    mark[torch.where(inside, s["table"].long(), s["pages"])] = True
    return mark[:-1], inside


def _free(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        r = api.paged_kv_free(s["gone"], s["kv_lens"], s["free"], s["head"], s["table"],
                              page_size=s["page"], num_pages=s["pages"], status=s["status"])
        return [s["free"], r.seq_lens, r.free_head]
    left = s["kv_lens"].clone()
    left[s["gone"].long()] = 0
    freed = _marks(s, s["kv_lens"])[0] & ~_marks(s, left)[0]
    rank = freed.long().cumsum(0) - 1
    head = s["head"].long() - freed.sum()
    n = s["free"].numel()
    ids = torch.arange(s["pages"], dtype=torch.int32, device="cuda")
    room = torch.cat([s["free"], s["free"].new_zeros(1)])
    room[torch.where(freed, head + rank, n)] = ids
    s["free"].copy_(room[:n])
    return [s["free"], left, head.to(torch.int32)]


def _compact(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        r = api.paged_kv_compact(s["kv_lens"], s["free"], s["head"], s["table"], page_size=s["page"],
                                 num_pages=s["pages"], status=s["status"])
        api.paged_kv_copy(s["pools"], r.src_pages, r.dst_pages, count=r.num_moves, status=s["status"])
        return [r.block_tables, r.free_pages, r.src_pages, r.dst_pages, r.num_moves, s["k_pages"],
                s["v_pages"]]
    used, inside = _marks(s, s["kv_lens"])
    n = s["free"].numel()
    at = torch.arange(n, device="cuda")
    open_ = torch.zeros(s["pages"] + 1, dtype=torch.bool, device="cuda")
    open_[torch.where(at >= s["head"], s["free"].long(), s["pages"])] = True
    open_ = open_[:-1]
    both = used | open_
    low = both & (both.long().cumsum(0) <= used.sum())   # where the pages in use belong
    hole, mover = low & open_, used & ~low
    ids = torch.arange(s["pages"], dtype=torch.int32, device="cuda")
    moves = min(n, s["pages"])
    src, dst = (torch.full((moves + 1,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    src[torch.where(mover, mover.long().cumsum(0) - 1, moves)] = ids
    dst[torch.where(hole, hole.long().cumsum(0) - 1, moves)] = ids
    src, dst = src[:-1], dst[:-1]
    to = ids.clone()
    to[mover] = dst[:ids.numel()][(mover.long().cumsum(0) - 1)[mover]]
    table = torch.where(inside, to[s["table"].clamp(min=0).long()], s["table"])
    rest = both & ~low
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free[torch.where(rest, s["head"] + rest.long().cumsum(0) - 1, n)] = ids
    src = torch.where(torch.arange(moves, device="cuda") < mover.sum(), src, -1)
    dst = torch.where(src >= 0, dst, -1)
    _move(s, src, dst)
    return [table, free[:n], src, dst, mover.sum(dtype=torch.int32).reshape(1), s["k_pages"], s["v_pages"]]


def _prefix(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        return list(api.paged_prefix_decode_run(s["plan"], s["q"], s["k_pages"], s["v_pages"], s["table"]))
    L, Hkv, ps = s["q_len"], s["kv_heads"], s["page"]
    G = s["heads"] // Hkv
    outs, lses, b0 = [], [], 0
    for pages, b1 in zip(s["pre"], s["ends"]):
        n, N = b1 - b0, pages * ps
        # [Hkv, n, L G, D]
        q = s["q"][b0 * L:b1 * L].float().view(n, L, Hkv, G, D).permute(2, 0, 1, 3, 4).reshape(Hkv, n, L * G, D)
        shared = s["table"][b0, :pages].long()
        k, v = (p[shared].float().transpose(0, 1).reshape(Hkv, N, D) for p in (s["k_pages"], s["v_pages"]))
        a = torch.matmul(q.reshape(Hkv, -1, D), k.transpose(1, 2)).mul_(s["scale"])
        width = max(1, -(-max(s["kv_host"][b0:b1]) // ps) - pages)
        rest = s["table"][b0:b1, pages:pages + width].long()
        if rest.shape[1] < width:
            rest = torch.nn.functional.pad(rest, (0, width - rest.shape[1]), value=-1)
        at = N + torch.arange(width * ps, device="cuda")
        kv = s["kv_lens"][b0:b1].long()
        inside = (at[None, :] < kv[:, None])[None, :, :, None]
        k2, v2 = (torch.where(inside, p[rest.clamp(min=0)].float().permute(2, 0, 1, 3, 4).reshape(Hkv, n, -1, D), 0.0)
                  for p in (s["k_pages"], s["v_pages"]))
        c = torch.matmul(q, k2.transpose(2, 3)) * s["scale"]
        last = kv[:, None] - L + torch.arange(L, device="cuda") if s["causal"] else (kv[:, None] - 1).expand(n, L)
        seen = at[None, None, :] <= last[:, :, None]
        c = torch.where(seen.repeat_interleave(G, 1)[None], c, -math.inf)
        top = torch.maximum(a.amax(-1).view(Hkv, n, L * G), c.amax(-1))[..., None]
        a = a.sub_(top.view(Hkv, -1, 1)).exp_()
        c = torch.exp(c - top)
        total = a.sum(-1).view(Hkv, n, L * G, 1) + c.sum(-1, keepdim=True)
        o = (torch.matmul(a, v).view(Hkv, n, L * G, D) + torch.matmul(c, v2)) / total
        lse = (top + torch.log(total)).squeeze(-1) / math.log(2.0)
        outs.append(o.view(Hkv, n, L, G, D).permute(1, 2, 0, 3, 4).reshape(n * L, Hkv * G, D).to(s["q"].dtype))
        lses.append(lse.view(Hkv, n, L, G).permute(1, 2, 0, 3).reshape(n * L, Hkv * G))
        b0 = b1
    return [torch.cat(outs), torch.cat(lses)]


_RUN = {"rope": _rope, "fork": _fork, "free": _free, "compact": _compact, "prefix": _prefix}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    g = torch.Generator()
    g.manual_seed(0)
    op = case["op"]
    page_bytes = case.get("kv_heads", 0) * case["page"] * D * 2
    if op == "rope":
        T, n = case["tokens"] + case["pad"], case["tokens"]
        H, Hkv = case["heads"], case["kv_heads"]
        return {"bytes": T * H * D * 4 + n * Hkv * D * 8 + 4 * case["axes"] * T + 8 * T,
                "flops": 3.0 * case["rotary"] * (T * H + n * Hkv)}
    if op == "fork":
        kv = _lens(case, g, case["parents"])
        mine = kv[torch.arange(case["forks"]) % case["parents"]]
        entries = float(((mine + case["page"] - 1) // case["page"]).sum())
        read = float(((kv + case["page"] - 1) // case["page"]).sum())
        tails = int((mine % case["page"] > 0).sum())
        return {"bytes": 4 * (read + entries) + 8 * case["batch"] + 20 * case["forks"] + tails * page_bytes * 4,
                "flops": 0.0}
    if op in ("free", "compact"):
        kv = _lens(case, g, case["batch"])
        width = -(-max(case["kv_hi"], 1) // case["page"]) + 1
        table, used = _family_tables(kv, case["page"], case["family"], width)
        entries = float((table >= 0).sum())
        if op == "free":   # half the released pages or so go back
            return {"bytes": 4 * entries + 8 * case["batch"] + 4 * case["rows"] * (1 + used / (2 * case["batch"])),
                    "flops": 0.0}
        pages = _pool_pages(case, kv)
        moves = used * (1 - used / pages)
        return {"bytes": 4 * (entries + table.numel()) + 8 * (pages - used) + 4 * case["batch"] + 8 * pages
                + moves * page_bytes * 4, "flops": 0.0}
    pre, group, suf = _prefix_lens(case, g)
    ps, L, H, B = case["page"], case["q_len"], case["heads"], case["batch"]
    keys = float(pre.sum()) * ps + float(suf.sum())
    pairs = float((pre[group] * ps + suf).sum()) * L - (B * L * (L - 1) / 2 if case["causal"] else 0)
    return {"bytes": keys * case["kv_heads"] * D * 4 + B * L * H * (D * 4 + 4) + 4 * keys / ps,
            "flops": 4.0 * D * H * pairs}


# ---- 64 bits, one request at a time ---------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op in ("free", "fork", "compact"):
        return None   # whole numbers, and pages copied as they are
    s = prepare(case, seed)
    if op == "rope":
        rd, half = case["rotary"], case["rotary"] // 2
        first = 0
        turned = [x.double() for x in (s["q"], s["k"])]
        for axis, count in enumerate(s["sections"]):
            for j in range(first, first + count):
                angle = s["pos"][axis].double() * case["base"] ** (-j / half)
                i0, i1 = (j, j + half) if case["pairs"] == "halves" else (2 * j, 2 * j + 1)
                z = torch.polar(torch.ones_like(angle), angle)[:, None]
                for x, y in zip((s["q"], s["k"]), turned):
                    w = torch.complex(x[..., i0].double(), x[..., i1].double()) * z
                    y[..., i0], y[..., i1] = w.real, w.imag
            first += count
        assert 2 * first == rd
        pools = []
        n = case["tokens"]
        slots = s["slots"][:n]
        for pool, rows in ((s["k_pages"], turned[1]), (s["v_pages"], s["v"].double())):
            flat = pool.double().transpose(1, 2).flatten(0, 1)
            flat[slots] = rows[:n]
            pools.append(flat.view(pool.shape[0], pool.shape[2], pool.shape[1], D).transpose(1, 2))
        return [turned[0], *pools]
    L, H, Hkv, ps = s["q_len"], s["heads"], s["kv_heads"], s["page"]
    G = H // Hkv
    out = torch.empty((s["q"].shape[0], H, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["q"].shape[0], H), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["kv_host"]):
        ids = s["table"][b, :-(-n // ps)].long()
        for h in range(Hkv):
            k, v = (p[ids, h].reshape(-1, D)[:n].double() for p in (s["k_pages"], s["v_pages"]))
            for i in range(L):
                m = n - L + i + 1 if s["causal"] else n
                row, at = b * L + i, slice(h * G, (h + 1) * G)
                x = s["q"][row, at].double() @ k[:m].T * s["scale"]
                lse[row, at] = torch.logsumexp(x, 1) / math.log(2.0)
                out[row, at] = torch.softmax(x, 1) @ v[:m]
    return [out, lse]
