"""Plain 64-bit latent attention and page bookkeeping for the latent tests, with the
error bounds that the kernels' number formats allow.

Bounds, per output element, with u(t) = finfo(t).eps / 2 the rounding of a format t:

* a score s = scale * sum q.k is summed in 32 bits over D products: at most
  D * 2^-24 * scale * sum |q.k| off (ds below, the largest over the row's keys);
* a weight p is off by a factor e^(2 ds) at most through the scores (numerator and sum),
  and is rounded to the input format before it meets the values: u(in);
* the values are summed in 32 bits in steps of 16 keys: (n / 16 + 32) * 2^-23;
  all three scale with A = sum p |v| / sum p;
* the result is rounded to its own format: u(out) * |o|.

The LSE is off by ds * log2(e) through the scores and by n / 16 + 64 roundings of 32
bits through the sum and the exponentials.
"""
import math

import torch


def u(dtype):
    return torch.finfo(dtype).eps / 2


def attention_rows(q, k, v, scale, out_scale, in_dtype, out_dtype):
    """q [H, D], k [n, D] or [H, n, D], v alike, all double.  Returns (o, lse, o bound,
    lse bound) of one query row; no keys give zeros and -inf."""
    H, n = q.shape[0], k.shape[-2]
    dv = v.shape[-1]
    if n == 0:
        z = torch.zeros((H, dv), dtype=torch.float64, device=q.device)
        return z, torch.full((H,), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0]
    if k.dim() == 2:
        k, v = k.expand(H, *k.shape), v.expand(H, *v.shape)
    s = torch.einsum("hd,hnd->hn", q, k) * scale
    ds = (torch.einsum("hd,hnd->hn", q.abs(), k.abs()).amax(1) * abs(scale) * q.shape[1] * 2 ** -24)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    o = torch.einsum("hn,hnd->hd", p, v) * out_scale
    A = torch.einsum("hn,hnd->hd", p, v.abs()) * abs(out_scale)
    rel = u(in_dtype) + 2 * ds + (n / 16 + 32) * 2 ** -23
    ob = A * rel[:, None]
    ob = ob + u(out_dtype) * (o.abs() + ob)
    lse = lse / math.log(2)
    lb = ds / math.log(2) + (n / 16 + 64) * 2 ** -24 + lse.abs() * 2 ** -22
    return o, lse, ob, lb


def ref_decode(q, pages, table, kv_lens, qo, dl, scale, causal, out_scale, out_dtype):
    """Absorbed decode of packed rows qo[b] .. qo[b + 1]."""
    ps = pages.shape[1]
    res = [[], [], [], []]
    for b, n in enumerate(kv_lens):
        ids = table[b, : -(-n // ps)].long()
        rows = pages[ids].flatten(0, 1)[:n].double()
        L = qo[b + 1] - qo[b]
        for i in range(L):
            m = max(0, n - L + i + 1) if causal else n
            got = attention_rows(q[qo[b] + i].double(), rows[:m], rows[:m, :dl], scale, out_scale,
                                 q.dtype, out_dtype)
            for r, x in zip(res, got):
                r.append(x)
    return [torch.stack(r) for r in res]


def ref_prefill(q, k, rope, v, qo, ko, scale, causal, out_scale, out_dtype, rows=None):
    """Expanded prefill; ``rows``: packed query rows to compute (default all)."""
    res = [[], [], [], []]
    picked = []
    for b in range(len(qo) - 1):
        lq, lk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        kk = torch.cat([k[ko[b]:ko[b + 1]].double(),
                        rope[ko[b]:ko[b + 1], None].double().expand(-1, k.shape[1], -1)], -1)
        kk, vv = kk.transpose(0, 1), v[ko[b]:ko[b + 1]].double().transpose(0, 1)
        for i in range(lq):
            if rows is not None and qo[b] + i not in rows:
                continue
            m = lk - lq + i + 1 if causal else lk
            got = attention_rows(q[qo[b] + i].double(), kk[:, :m], vv[:, :m], scale, out_scale,
                                 q.dtype, out_dtype)
            picked.append(qo[b] + i)
            for r, x in zip(res, got):
                r.append(x)
    return picked, [torch.stack(r) for r in res]


def assert_within(out, lse, ref):
    o, l, ob, lb = ref
    err = (out.double() - o).abs()
    assert bool((err <= ob).all()), (
        f"O off by {float(err.max()):.3g}, {float((err / ob.clamp(min=1e-30)).max()):.3g} of the "
        f"bound, first at {torch.nonzero(~(err <= ob))[:3].tolist()}")
    if lse is not None:
        empty = l == -math.inf
        assert bool((lse.double()[empty] == -math.inf).all())
        lerr = (lse.double() - l)[~empty].abs()
        assert bool((lerr <= lb[~empty]).all()), f"LSE off by {float(lerr.max()):.3g}"


def ref_tables(kv, new, free, head, table, ps, num_slots):
    """The page bookkeeping on host lists; None when the step does not fit."""
    table = [list(r) for r in table]
    slots, qo, pos_in_free = [], [0], head
    for b, (n, w) in enumerate(zip(kv, new)):
        if n < 0 or w < 0 or n + w > len(table[b]) * ps:
            return None
        for j in range(-(-n // ps), -(-(n + w) // ps)):
            if pos_in_free >= len(free) or head < 0:
                return None
            table[b][j] = free[pos_in_free]
            pos_in_free += 1
        slots += [table[b][x // ps] * ps + x % ps for x in range(n, n + w)]
        qo.append(qo[-1] + w)
    if len(slots) > num_slots or head < 0 or head > len(free):
        return None
    slots += [-1] * (num_slots - len(slots))
    return table, [n + w for n, w in zip(kv, new)], qo, slots, pos_in_free
