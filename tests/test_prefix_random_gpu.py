"""Decode behind shared prefixes over drawn batches, against 64-bit attention, and batches at the
ends of its range."""

import random

import pytest
import torch

from paged_kv_attention_32_gb300 import api
from tests import prefix_ref as ref
from tests.test_prefix_gpu import check, close, make, plan_of, table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(24))
def test_drawn_batches(seed):
    """Groups of none to many requests, prefixes of none to many pages, packed rows, masks, types,
    sinks, scales, few and many SMs: every combination has to hold."""
    r = random.Random(seed)
    ps = r.choice([16, 16, 32, 48, 64, 80, 128])
    kv_heads = r.choice([1, 2, 3, 8])
    heads = kv_heads * r.choice([1, 2, 4, 5, 7, 8, 16])
    causal = r.random() < 0.5
    groups, q_lens = [], []
    for _ in range(r.randint(1, 5)):
        own, pages = [], r.choice([0, 1, 2, 7, 40])
        for _ in range(r.choice([0, 1, 2, 3, 9, 20])):
            n = r.choice([1, 1, 1, 2, 4, 9])
            q_lens.append(n)
            # own keys: none where the mask allows it, a page's end, odd numbers
            least = (n - 1 if causal else 0) if pages else n
            own.append(least + r.choice([0, 1, ps - 1, ps, 3 * ps + 5, r.randint(0, 700)]))
        groups.append((pages, own))
    if not q_lens:
        groups, q_lens = [(3, [0, 5])], [1, 1]
    c = make(groups, heads=heads, kv_heads=kv_heads, ps=ps, q_lens=q_lens, seed=seed, spare_cols=r.randint(0, 3),
             dtype=r.choice([torch.bfloat16, torch.float16]), scale=r.choice([None, 0.3, -0.05]))
    kw = dict(causal=causal, out_dtype=r.choice([None, torch.float32]), bmm2_scale=r.choice([1.0, 2.5]))
    p = plan_of(c, num_sms=r.choice([0, 0, 1, 5, 200]), **kw)
    some = any(len(own) > 1 and pages > 0 for pages, own in groups)
    check(c, plan=p, pieces=some, sinks=torch.randn(heads, device="cuda") if r.random() < 0.3 else None, **kw)


def compared(c, rows, out, lse, causal=False):
    """The given requests' rows against 64 bits."""
    at = [x for b in rows for x in range(c["qo"][b], c["qo"][b + 1])]
    qo = [0]
    for b in rows:
        qo.append(qo[-1] + c["qo"][b + 1] - c["qo"][b])
    want = ref.decode(c["q"][at], c["k"], c["v"], [c["tables"][b] for b in rows], [c["kv"][b] for b in rows], qo,
                      causal=causal, scale=c["scale"])
    close((out[at], lse[at]), want, c["v"], c["dtype"], c["dtype"])


def test_thousands_of_requests():
    """3000 requests of few own keys behind one prefix and 1000 behind none; samples of them compared, and all
    with the decode that shares nothing."""
    c = make([(9, [1 + i % 40 for i in range(3000)]), (0, [1 + i % 90 for i in range(1000)])], heads=8, kv_heads=2, ps=16)
    p = plan_of(c)
    out, lse = api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], table(c))
    p.check()
    compared(c, [0, 1, 77, 2047, 2999, 3000, 3999], out, lse)
    plain = plan_of(c, min_shared_bytes=1 << 60)
    want, want_lse = api.paged_prefix_decode_run(plain, c["q"], c["k"], c["v"], table(c))
    # both within the bound that the 64-bit comparison uses: of the mean of |v| and of the output
    top, eps = float(c["v"].abs().max()), torch.finfo(c["dtype"]).eps / 2
    bound = 2 * (eps * want.double().abs() + (eps + 2.0 ** -18) * top)
    assert bool(((out.double() - want.double()).abs() <= bound).all())
    assert bool(((lse - want_lse).abs() <= 2 * (2.0 ** -18 * want_lse.abs().clamp(min=1) + 2.0 ** -16)).all())


def test_long_own_keys_and_a_short_prefix():
    c = make([(1, [30000, 3, 9000])], heads=8, kv_heads=1, ps=16, seed=1)
    check(c)


def test_many_rows_of_one_request():
    """Rows that a verified or chunked step packs: 600 of one request, causal."""
    c = make([(30, [700, 650])], heads=8, kv_heads=2, ps=32, q_lens=[600, 3], seed=2)
    check(c, causal=True)


def test_heads_that_share_their_queries():
    """Query heads that are one row expanded, tokens likewise: strides of zero are read, never written."""
    c = make([(30, [70, 65, 9])], heads=8, kv_heads=2, ps=16, seed=3)
    c["q"] = c["q"][:, :1].expand(-1, 8, -1)
    check(c)
    c["q"] = c["q"][:1].expand(3, -1, -1)
    check(c)
