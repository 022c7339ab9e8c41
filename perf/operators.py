"""Cases of the latent-attention serving path: page tables and slot maps built on the
GPU, new latent rows appended to the paged cache, absorbed decode over that cache and
expanded prefill.

One cached token of latent attention is a row of ``dl`` latent values, shared by every
head as key and value, followed by ``dr`` rotary key values.  ``run`` computes each
operator either in elementary torch operations (32-bit, rounded once) or, with ``own``,
through the package's entry points.
"""

import math

import torch

own = False

DN, DV, DR = 128, 128, 64   # expanded head: key part without rotation, value, rotary part
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decode step of a 64-request batch: every request gains a token, one in
        # sixteen needs a new page
        dict(name="tables_step_b64", op="tables", batch=64, page=16, kv_lo=512, kv_hi=8191,
             new_lo=1, new_hi=1, slots=64),
        # a scheduler's mixed step: many requests, ragged chunks, some of them idle, the
        # slot map padded to the step's token budget
        dict(name="tables_mixed_b1024", op="tables", batch=1024, page=32, kv_lo=0, kv_hi=4096,
             new_lo=0, new_hi=63, slots=65536),
        # one decode step: 64 tokens to scattered pages
        dict(name="append_step_t64", op="append", tokens=64, pad=0, dl=512, page=16, pages=4096,
             dtype="bf16"),
        # a long prefill chunk, its padded tail skipped
        dict(name="append_chunk_t32768", op="append", tokens=32000, pad=768, dl=512, page=64,
             pages=1024, dtype="bf16"),
        # the smallest decode: a few short requests, bound by latency
        dict(name="decode_tiny_b4", op="decode", batch=4, heads=8, dl=256, page=16, kv_lo=1,
             kv_hi=300, first=0, q_len=1, causal=False, dtype="bf16"),
        # an ordinary serving batch with ragged lengths
        dict(name="decode_ragged_b64_h32", op="decode", batch=64, heads=32, dl=512, page=16,
             kv_lo=512, kv_hi=8192, first=0, q_len=1, causal=False, dtype="bf16"),
        # one long context among ordinary ones
        dict(name="decode_long_b16_h64", op="decode", batch=16, heads=64, dl=512, page=32,
             kv_lo=1024, kv_hi=4096, first=131072, q_len=1, causal=False, dtype="bf16"),
        # verification of drafted tokens: four causal query rows a request
        dict(name="decode_spec_b32_h64_q4", op="decode", batch=32, heads=64, dl=512, page=16,
             kv_lo=2048, kv_hi=16384, first=0, q_len=4, causal=True, dtype="f16"),
        # many heads on one GPU
        dict(name="decode_wide_b64_h128", op="decode", batch=64, heads=128, dl=512, page=64,
             kv_lo=512, kv_hi=8192, first=0, q_len=1, causal=False, dtype="bf16"),
        # the smallest prefill: three short prompts
        dict(name="prefill_tiny_b3", op="prefill", batch=3, heads=4, q_lo=1, q_hi=130, past=0,
             causal=True, dtype="bf16"),
        # a batch of ragged prompts
        dict(name="prefill_ragged_b8_h32", op="prefill", batch=8, heads=32, q_lo=512, q_hi=4096,
             past=0, causal=True, dtype="bf16"),
        # the last chunk of long prompts: bottom-right causal rows behind cached keys
        dict(name="prefill_chunk_b2_h32", op="prefill", batch=2, heads=32, q_lo=1000, q_hi=1024,
             past=7168, causal=True, dtype="f16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode", "decode", "prefill", "prefill"])
    if op == "tables":
        batch, new_hi = _log(rng, 1, 2048), _log(rng, 1, 64)
        new_lo = rng.choice([0, 1])
        need = batch * new_hi
        return dict(op=op, batch=batch, page=rng.choice([8, 16, 32, 48, 64, 128]),
                    kv_lo=rng.choice([0, 1, 100]), kv_hi=_log(rng, 100, 8191), new_lo=new_lo,
                    new_hi=new_hi, slots=need + rng.choice([0, 1, need // 3]))
    if op == "append":
        page = rng.choice([8, 16, 32, 64])
        tokens = _log(rng, 1, 30000)
        pad = rng.choice([0, 0, 1 + tokens // 7])
        return dict(op=op, tokens=tokens, pad=pad, dl=rng.choice([256, 512]), page=page,
                    pages=-(-tokens // page) + _log(rng, 8, 512),
                    dtype=rng.choice(["bf16", "f16"]))
    if op == "decode":
        heads = rng.choice([1, 5, 8, 16, 20, 32, 40, 64, 96, 128])
        q_len = rng.choice([1, 1, 1, 2, 3, 5])
        kv_hi = _log(rng, 1, 8192)
        batch = _log(rng, 1, 64)
        batch = max(1, min(batch, 64 * 128 // (heads * q_len)))   # within the widest listed case
        return dict(op=op, batch=batch, heads=heads, dl=rng.choice([256, 512, 512]),
                    page=rng.choice([8, 16, 32, 48, 64, 128]), kv_lo=rng.choice([0, 1, kv_hi // 2]),
                    kv_hi=kv_hi, first=rng.choice([0, 0, 0, _log(rng, 1, 32768)]), q_len=q_len,
                    causal=q_len > 1 or rng.random() < 0.3, dtype=rng.choice(["bf16", "bf16", "f16"]))
    q_hi = _log(rng, 1, 2600)
    return dict(op=op, batch=_log(rng, 1, 6), heads=rng.choice([1, 3, 8, 16, 20, 32]),
                q_lo=rng.choice([1, max(1, q_hi // 3), q_hi]), q_hi=q_hi,
                past=rng.choice([0, 0, _log(rng, 1, 2000)]), causal=rng.random() < 0.7,
                dtype=rng.choice(["bf16", "bf16", "f16"]))


# ---- inputs -------------------------------------------------------------------

def _gens(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    d = torch.Generator(device="cuda")
    d.manual_seed(seed + 1)
    return g, d


def _lens(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)


def _decode_lens(case, g):
    """The case's own key lengths, the requests in an order of ``g``'s."""
    own_lens = torch.Generator()
    own_lens.manual_seed(0)
    kv = _lens(own_lens, case["kv_lo"], max(case["kv_lo"], case["kv_hi"]), case["batch"])
    if case["first"]:
        kv[0] = case["first"]
    return kv[torch.randperm(case["batch"], generator=g)]


def _prefill_lens(case, g):
    own_lens = torch.Generator()
    own_lens.manual_seed(0)
    q = _lens(own_lens, case["q_lo"], case["q_hi"], case["batch"])
    q = q[torch.randperm(case["batch"], generator=g)]
    return q, q + case["past"]


def prepare(case, seed):
    g, d = _gens(seed)
    s = dict(case)
    op = case["op"]
    if op == "tables":
        B, ps = case["batch"], case["page"]
        kv, new = _lens(g, case["kv_lo"], case["kv_hi"], B), _lens(g, case["new_lo"], case["new_hi"], B)
        have, need = (kv + ps - 1) // ps, (kv + new + ps - 1) // ps
        width = -(-(case["kv_hi"] + case["new_hi"]) // ps) + 1
        pool = B * (width - 1) + 37
        perm = torch.randperm(pool, generator=g, dtype=torch.int64).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32)
        inside = torch.arange(width)[None, :] < have[:, None]
        used = int(have.sum())
        table[inside] = perm[:used]
        head = int(torch.randint(0, 8, (1,), generator=g))
        free = torch.cat([torch.full((head,), -1, dtype=torch.int32), perm[used:]])
        s.update(kv_lens=kv.to(torch.int32).cuda(), new_lens=new.to(torch.int32).cuda(),
                 table=table.cuda(), free=free.cuda(),
                 head=torch.tensor([head], dtype=torch.int32, device="cuda"),
                 status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    elif op == "append":
        dt, T = _DTYPES[case["dtype"]], case["tokens"] + case["pad"]
        n = case["pages"] * case["page"]
        pages = torch.randn((case["pages"], case["page"], case["dl"] + DR), generator=d,
                            device="cuda", dtype=dt)
        rows = torch.randn((T, case["dl"] + DR), generator=d, device="cuda", dtype=dt)
        # tokens fill pages in order, the pages are scattered over the pool
        order = torch.randperm(case["pages"], generator=g, dtype=torch.int64)
        t = torch.arange(case["tokens"], dtype=torch.int64)
        if case["tokens"] <= 64:   # a decode step: each token in a page of its own
            slots = order[t % case["pages"]] * case["page"] + (t // case["pages"])
        else:
            slots = order[t // case["page"]] * case["page"] + t % case["page"]
        slots = torch.cat([slots, torch.full((case["pad"],), -1, dtype=torch.int64)])
        assert int(slots.max()) < n
        s.update(pages=pages, latent=rows[:, :case["dl"]], rope=rows[:, case["dl"]:],
                 slots=slots.cuda(), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    elif op == "decode":
        dt, B, H, ps = _DTYPES[case["dtype"]], case["batch"], case["heads"], case["page"]
        kv = _decode_lens(case, g)
        need = (kv + ps - 1) // ps
        width, used = max(1, int(need.max())), int(need.sum())
        pool = used + 7
        perm = torch.randperm(pool, generator=g, dtype=torch.int64).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32)
        table[torch.arange(width)[None, :] < need[:, None]] = perm[:used]
        D = case["dl"] + DR
        pages = torch.randn((pool, ps, D), generator=d, device="cuda", dtype=dt)
        q = torch.randn((B * case["q_len"], H, D), generator=d, device="cuda", dtype=dt)
        s.update(pages=pages, q=q, table=table.cuda(), kv_lens=kv.to(torch.int32).cuda(),
                 scale=1.0 / math.sqrt(D))
        if own:
            from paged_kv_attention_32_gb300 import api
            s["plan"] = api.paged_latent_decode_plan(
                kv.to(torch.int32), num_heads=H, page_size=ps, max_pages_per_seq=width,
                num_pages=pool, latent_dim=case["dl"], rope_dim=DR, q_len=case["q_len"],
                causal=case["causal"], scale=s["scale"], return_lse=True, dtype=dt)
    else:
        dt, H = _DTYPES[case["dtype"]], case["heads"]
        lq, lk = _prefill_lens(case, g)
        zero = torch.zeros(1, dtype=torch.int64)
        qo = torch.cat([zero, lq.cumsum(0)]).to(torch.int32)
        ko = torch.cat([zero, lk.cumsum(0)]).to(torch.int32)
        q = torch.randn((int(qo[-1]), H, DN + DR), generator=d, device="cuda", dtype=dt)
        kv = torch.randn((int(ko[-1]), H, DN + DV), generator=d, device="cuda", dtype=dt)
        rope = torch.randn((int(ko[-1]), DR), generator=d, device="cuda", dtype=dt)
        s.update(q=q, k=kv[..., :DN], v=kv[..., DN:], rope=rope, qo=qo.cuda(), ko=ko.cuda(),
                 lq_max=int(lq.max()), lk_max=int(lk.max()), scale=1.0 / math.sqrt(DN + DR))
        if own:
            from paged_kv_attention_32_gb300 import api
            s["plan"] = api.batch_latent_prefill_plan(
                qo, ko, num_heads=H, causal=case["causal"], sm_scale=s["scale"], return_lse=True,
                dtype=dt)
    return s


# ---- one pass -------------------------------------------------------------------

def run(s):
    return _RUN[s["op"]](s)


def _tables(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        r = api.paged_kv_tables(s["kv_lens"], s["new_lens"], s["free"], s["head"], s["table"],
                                page_size=s["page"], num_slots=s["slots"], status=s["status"])
        return [s["table"], r.seq_lens, r.qo_indptr, r.slot_map, r.free_head]
    ps, kv, new, table = s["page"], s["kv_lens"].long(), s["new_lens"].long(), s["table"]
    have, need = (kv + ps - 1) // ps, (kv + new + ps - 1) // ps
    grow = need - have
    base = s["head"].long() + grow.cumsum(0) - grow
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (j >= have[:, None]) & (j < need[:, None])
    src = (base[:, None] + j - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][src], table)
    ends = new.cumsum(0)
    t = torch.arange(s["slots"], device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    live = b < kv.numel()
    b = b.clamp(max=kv.numel() - 1)
    pos = kv[b] + t - (ends - new)[b]
    page = (pos // ps).clamp(0, table.shape[1] - 1)
    slot = table[b, page].long() * ps + pos % ps
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    return [table, (kv + new).to(torch.int32), torch.cat([zero, ends.to(torch.int32)]),
            torch.where(live, slot, -1), (s["head"] + grow.sum()).to(torch.int32)]


def _append(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        return api.paged_latent_append(s["latent"], s["rope"], s["slots"], s["pages"],
                                       status=s["status"])
    keep = s["slots"] >= 0
    rows = torch.cat([s["latent"], s["rope"]], 1)
    s["pages"].view(-1, rows.shape[1])[s["slots"][keep]] = rows[keep]
    return s["pages"]


def _softmax(score, seen):
    """(weights, base-2 LSE) of masked scores; a row that sees nothing has zero weights
    and an LSE of -inf."""
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1) / math.log(2.0)
    return p / torch.where(total == 0, 1.0, total), lse


def _decode(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        return list(api.paged_latent_decode_run(s["plan"], s["q"], s["pages"], s["table"]))
    B, H, L, dl = s["batch"], s["heads"], s["q_len"], s["dl"]
    rows = s["pages"][s["table"].clamp(min=0).long()].flatten(1, 2)
    n = rows.shape[1]
    kv = s["kv_lens"].long()
    inside = torch.arange(n, device="cuda")[None, :] < kv[:, None]
    rows = torch.where(inside[..., None], rows.float(), 0.0)
    q = s["q"].float().view(B, L * H, -1)
    score = torch.matmul(q, rows.transpose(1, 2)).view(B, L, H, n) * s["scale"]
    last = kv[:, None] - L + torch.arange(L, device="cuda") if s["causal"] else \
        (kv[:, None] - 1).expand(B, L)
    seen = torch.arange(n, device="cuda") <= last[:, :, None, None]
    p, lse = _softmax(score, seen)
    out = torch.matmul(p.view(B, L * H, n), rows[..., :dl])
    return [out.view(B * L, H, dl).to(s["q"].dtype), lse.reshape(B * L, H)]


def _prefill(s):
    if own:
        from paged_kv_attention_32_gb300 import api
        return list(api.batch_latent_prefill_run(s["plan"], s["q"], s["k"], s["rope"], s["v"]))
    H, nq, nk = s["heads"], s["lq_max"], s["lk_max"]
    qo, ko = s["qo"].long(), s["ko"].long()
    lq, lk = qo.diff(), ko.diff()
    iq, ik = torch.arange(nq, device="cuda"), torch.arange(nk, device="cuda")
    # requests padded to the longest one
    at_q = (qo[:-1, None] + torch.minimum(iq, (lq[:, None] - 1).clamp(min=0)))
    at_k = (ko[:-1, None] + torch.minimum(ik, (lk[:, None] - 1).clamp(min=0)))
    k = torch.cat([s["k"], s["rope"][:, None, :].expand(-1, H, -1)], -1)
    q = s["q"][at_q].float().transpose(1, 2)
    k = k[at_k].float().transpose(1, 2)
    v = s["v"][at_k].float().transpose(1, 2)
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    seen = (ik < lk[:, None])[:, None, :]
    if s["causal"]:
        seen = seen & (ik <= (lk - lq)[:, None, None] + iq[None, :, None])
    p, lse = _softmax(score, seen[:, None])
    out = torch.matmul(p, v).transpose(1, 2)
    live = (iq < lq[:, None])
    return [out[live].to(s["q"].dtype), lse.transpose(1, 2)[live]]


_RUN = {"tables": _tables, "append": _append, "decode": _decode, "prefill": _prefill}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    g = torch.Generator()
    g.manual_seed(0)
    op = case["op"]
    if op == "tables":
        B, ps = case["batch"], case["page"]
        kv = (case["kv_lo"] + case["kv_hi"]) / 2
        new = (case["new_lo"] + case["new_hi"]) / 2
        pages = B * new / ps   # taken from the free list and written to the table
        return {"bytes": B * (4 * 4) + 8 * pages + 8 * case["slots"] + (4 * B if kv else 0),
                "flops": 0.0}
    if op == "append":
        row = 2 * (case["dl"] + DR)
        return {"bytes": case["tokens"] * 2 * row + 8 * (case["tokens"] + case["pad"]), "flops": 0.0}
    if op == "decode":
        n = float(_decode_lens(case, g).sum())
        rows = case["batch"] * case["q_len"] * case["heads"]
        D = case["dl"] + DR
        return {"bytes": n * D * 2 + rows * (D * 2 + case["dl"] * 2 + 4) + 4 * n / case["page"],
                "flops": 2.0 * n * case["q_len"] * case["heads"] * (D + case["dl"])}
    lq, lk = _prefill_lens(case, g)
    lq, lk = lq.double(), lk.double()
    pairs = lq * lk - (lq * (lq - 1) / 2 if case["causal"] else 0)
    H = case["heads"]
    tokens_q, tokens_k = float(lq.sum()), float(lk.sum())
    return {"bytes": tokens_q * H * ((DN + DR) * 2 + DV * 2 + 4) + tokens_k * (H * (DN + DV) + DR) * 2,
            "flops": 2.0 * float(pairs.sum()) * H * (DN + DR + DV)}


# ---- 64 bits, one request at a time ---------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None   # whole numbers
    s = prepare(case, seed)
    if op == "append":
        n = case["tokens"]
        pages = s["pages"].double().flatten(0, 1)
        pages[s["slots"][:n], :case["dl"]] = s["latent"][:n].double()
        pages[s["slots"][:n], case["dl"]:] = s["rope"][:n].double()
        return pages.view(s["pages"].shape)
    inf = float("inf")
    if op == "decode":
        L, H, dl = s["q_len"], s["heads"], s["dl"]
        out = torch.zeros((s["batch"] * L, H, dl), dtype=torch.float64, device="cuda")
        lse = torch.full((s["batch"] * L, H), -inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["kv_lens"].tolist()):
            ids = s["table"][b, : -(-n // s["page"])].long()
            keys = s["pages"][ids].reshape(-1, dl + DR)[:n].double()
            for i in range(L):
                m = min(n, n - L + i + 1) if s["causal"] else n
                if m > 0:
                    x = s["q"][b * L + i].double() @ keys[:m].T * s["scale"]
                    lse[b * L + i] = torch.logsumexp(x, 1) / math.log(2.0)
                    out[b * L + i] = torch.softmax(x, 1) @ keys[:m, :dl]
        return [out, lse]
    H = s["heads"]
    out = torch.zeros((s["q"].shape[0], H, DV), dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], H), -inf, dtype=torch.float64, device="cuda")
    qo, ko = s["qo"].tolist(), s["ko"].tolist()
    for b in range(s["batch"]):
        nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        rope = s["rope"][ko[b]:ko[b + 1]].double()
        for h in range(H):
            q = s["q"][qo[b]:qo[b + 1], h].double()
            k = s["k"][ko[b]:ko[b + 1], h].double()
            x = (q[:, :DN] @ k.T + q[:, DN:] @ rope.T) * s["scale"]
            if s["causal"]:
                x = x.masked_fill(~torch.ones_like(x, dtype=torch.bool).tril(nk - nq), -inf)
            lse[qo[b]:qo[b + 1], h] = torch.logsumexp(x, 1) / math.log(2.0)
            out[qo[b]:qo[b + 1], h] = torch.softmax(x, 1) @ s["v"][ko[b]:ko[b + 1], h].double()
    return [out, lse]
