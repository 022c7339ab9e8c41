"""Decode behind long shared prefixes within the error of its roundings alone, which a tile of values read from
the wrong page or stage would pass many times over."""

import pytest
import torch

from paged_kv_attention_32_gb300 import api
from tests import prefix_bounds as bounds
from tests.test_prefix_gpu import make, plan_of, table

pytestmark = pytest.mark.gpu


def within(c, plan, causal=False, out_dtype=torch.float32):
    out, lse = api.paged_prefix_decode_run(plan, c["q"], c["k"], c["v"], table(c))
    plan.check()
    prefix, own = plan.export()
    piece = max([64 * (x[4] - x[3]) for x in prefix] + [16 * (x[4] - x[3]) for x in own])
    want, want_lse, allowed = bounds.decode(c["q"], c["k"], c["v"], c["tables"], c["kv"], c["qo"], causal=causal,
                                            scale=c["scale"], dtype=c["dtype"], out_dtype=out_dtype, piece=piece)
    err = (out.double() - want).abs()
    assert bool((err <= allowed).all()), f"up to {float((err / allowed).max())} times what is allowed"
    assert bool(((lse.double() - want_lse).abs() <= 2.0 ** -18 * want_lse.abs().clamp(min=1) + 2.0 ** -16).all())
    return want, allowed


@pytest.mark.parametrize("out_dtype", [torch.float32, None])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sms", [0, 2])
@pytest.mark.parametrize("pages,ps", [(1, 16), (7, 16), (100, 16), (60, 48), (100, 64), (30, 256)])
def test_prefixes(pages, ps, sms, dtype, out_dtype):
    c = make([(pages, [20, 1, 0, 33, 70, 300])], heads=8, kv_heads=2, ps=ps, dtype=dtype, seed=pages)
    p = plan_of(c, num_sms=sms, out_dtype=out_dtype)
    assert p.info["shared"]
    within(c, p, out_dtype=out_dtype or dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("requests,q_len,kv_heads,sms,dense", [(3, 1, 8, 0, 0), (40, 2, 2, 0, 0), (40, 4, 2, 3, 1), (70, 1, 1, 1, 1)])
def test_rows_and_masks(dtype, requests, q_len, kv_heads, sms, dense):
    """Few rows and many, in both shapes of the prefix kernel, packed and causal."""
    c = make([(200, [q_len + 7 * i % 90 for i in range(requests)])], heads=8, kv_heads=kv_heads, ps=16, dtype=dtype,
             q_lens=[q_len] * requests, seed=requests)
    p = plan_of(c, num_sms=sms, out_dtype=torch.float32, causal=q_len > 1)
    assert p.info["dense"] == dense
    within(c, p, causal=q_len > 1)


@pytest.mark.parametrize("sms", [0, 4])
@pytest.mark.parametrize("ps,keys", [(16, 8192), (64, 65536)])
def test_values_that_name_their_tile(ps, keys, sms):
    """Values that are 1 or -1 for all of a tile of 64 keys and one dimension: one tile out of place would move
    half of the dimensions by twice its weight, and so past the bound, whichever way the roundings go."""
    c = make([(keys // ps, [0, 0, 0, 0])], heads=8, kv_heads=2, ps=ps, dtype=torch.float16, seed=9)
    ids = torch.tensor(c["tables"][0][:keys // ps], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    sign = (torch.randint(0, 2, (keys // 64, 2, 128), generator=g, device="cuda") * 2 - 1).half()
    c["v"][ids] = sign.repeat_interleave(64, 0).view(keys // ps, ps, 2, 128).transpose(1, 2).contiguous()
    c["q"] = c["q"] / 4   # weights near to each other
    want, allowed = within(c, plan_of(c, num_sms=sms, out_dtype=torch.float32))
    k = c["k"][ids].transpose(0, 1).reshape(2, keys, 128).double()
    for h in range(2):
        w = torch.softmax(c["q"][:, 4 * h:4 * h + 4].double() @ k[h].T * c["scale"], -1)
        lightest = w.view(*w.shape[:2], -1, 64).sum(-1).amin(-1)
        assert bool((lightest[..., None] > allowed[:, 4 * h:4 * h + 4]).all())
