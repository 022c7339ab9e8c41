"""Decodes over pools whose slots past a request's last key hold infinities and NaN, as freshly allocated
memory may: every kernel, planned and live lengths, against 64-bit attention over the keys alone."""

import pytest
import torch

from paged_kv_attention_32_gb300 import api
from tests import prefix_ref as ref
from tests.test_prefix_gpu import close, make, plan_of, table

pytestmark = pytest.mark.gpu


def poisoned(c, lens):
    """The pools, but for the first `lens` slots of each request, filled with infinities and NaN."""
    ps, pools = c["ps"], []
    keep = torch.zeros(c["k"].shape[0], ps, dtype=torch.bool, device="cuda")
    for row, n in zip(c["tables"], lens):
        at = torch.arange(n, device="cuda")
        keep[torch.tensor(row, device="cuda")[at // ps], at % ps] = True
    for pool, bad in ((c["k"], float("nan")), (c["v"], float("inf"))):
        rest = torch.full_like(pool, bad)
        rest[..., ::3] = -float("inf")
        pools.append(torch.where(keep[:, None, :, None], pool, rest))
    return pools


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mma_min_rows", [1, 9])
@pytest.mark.parametrize("heads,kv_heads,q_len", [(4, 4, 1), (8, 4, 1), (4, 2, 2), (8, 1, 1), (4, 1, 2)])
@pytest.mark.parametrize("live", [False, True])
def test_slots_past_the_last_key(dtype, mma_min_rows, heads, kv_heads, q_len, live):
    own = [q_len, 15, 16, 17, 40, 700, 1500]
    c = make([(0, own)], heads=heads, kv_heads=kv_heads, ps=32, q_lens=[q_len] * len(own), dtype=dtype, seed=heads)
    lens = [max(q_len, n - 1 - 9 * i) for i, n in enumerate(c["kv"])] if live else c["kv"]
    k, v = poisoned(c, lens)
    plan = api.paged_decode_plan(c["kv"], num_qo_heads=heads, num_kv_heads=kv_heads, page_size=32,
                                 max_pages_per_seq=c["width"], num_pages=k.shape[0], q_len=q_len, causal=q_len > 1,
                                 scale=c["scale"], return_lse=True, dtype=dtype, mma_min_rows=mma_min_rows,
                                 freeze_seq_lens=not live)
    assert plan.info["kernel"] == int(mma_min_rows == 1)
    now = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = api.paged_decode_run(plan, c["q"], k, v, table(c), seq_lens_kv=now if live else None)
    plan.check()
    want = ref.decode(c["q"], c["k"], c["v"], c["tables"], lens, c["qo"], causal=q_len > 1, scale=c["scale"])
    close(got, want, c["v"], dtype, dtype)


@pytest.mark.parametrize("mma_min_rows", [1, 9])
@pytest.mark.parametrize("min_shared_bytes", [0, 1 << 40])
@pytest.mark.parametrize("live", [False, True])
def test_slots_past_the_last_key_behind_a_prefix(mma_min_rows, min_shared_bytes, live):
    c = make([(3, [1, 70, 5, 300]), (0, [9])], heads=8, kv_heads=2, ps=16, seed=1)
    lens = [max(3 * 16 if b < 4 else 1, n - 4 * b) for b, n in enumerate(c["kv"])] if live else c["kv"]
    k, v = poisoned(c, lens)
    p = plan_of(c, min_shared_bytes=min_shared_bytes, mma_min_rows=mma_min_rows, freeze_seq_lens=not live)
    assert bool(p.info["shared"]) == (min_shared_bytes == 0)
    now = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = api.paged_prefix_decode_run(p, c["q"], k, v, table(c), seq_lens_kv=now if live else None)
    p.check()
    want = ref.decode(c["q"], c["k"], c["v"], c["tables"], lens, c["qo"], causal=False, scale=c["scale"])
    close(got, want, c["v"], c["dtype"], c["dtype"])
