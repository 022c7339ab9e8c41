"""Many keys of tiny weight beside one that holds nearly all of it, in f16, whose numbers end at
2^-24: together the tiny ones are what the output consists of where the large one's value is 0.

The bound is latent_ref's, which takes a weight's rounding as u(f16) of it, and for weights below
f16's normal range half a step, 2^-25, of weights whose largest is 2^7 at least (the kernels scale
them so): at most 2^-32 sum |v| of the row's keys."""
import math

import pytest
import torch

from latent_ref import ref_decode, ref_prefill
from paged_kv_attention_32_gb300 import api

pytestmark = pytest.mark.gpu

DEV, HF = "cuda", torch.float16


def assert_close(out, lse, ref, extra):
    o, l, ob, lb = ref
    err = (out.double() - o).abs()
    assert bool((err <= ob + extra).all()), (
        f"O off by {float(err.max()):.3g}, {float((err / (ob + extra)).max()):.3g} of the bound")
    assert bool(((lse.double() - l).abs() <= lb).all())


def exponents(n, at, g):
    """log2 of the keys' weights: 0 for key ``at``, -22 to -29 for the others."""
    x = -22 - 7 * torch.rand(n, generator=g, device=DEV)
    x[at] = 0
    return x.to(HF)


@pytest.mark.parametrize("at", [0, 10000, 19999])
@pytest.mark.parametrize("num_sms", [1, 152])
@pytest.mark.parametrize("heads", [16, 64, 128])
def test_decode_small_weights(heads, num_sms, at):
    n, dl, ps = 20000, 256, 64
    g = torch.Generator(device=DEV).manual_seed(at)
    rows = torch.zeros((n, dl + 64), dtype=HF, device=DEV)
    rows[:, :dl] = 0.5 + 0.5 * torch.rand((n, dl), generator=g, device=DEV)
    rows[at, : dl // 2] = 0
    rows[:, dl] = exponents(n, at, g)
    pages = torch.zeros((313, ps, dl + 64), dtype=HF, device=DEV)
    pages.view(-1, dl + 64)[:n] = rows
    table = torch.arange(313, dtype=torch.int32, device=DEV)[None]
    q = torch.zeros((1, heads, dl + 64), dtype=HF, device=DEV)
    q[..., dl] = 1
    plan = api.paged_latent_decode_plan([n], num_heads=heads, page_size=ps, max_pages_per_seq=313,
                                        num_pages=313, scale=math.log(2), latent_dim=dl, dtype=HF,
                                        out_dtype=torch.float32, return_lse=True, num_sms=num_sms)
    out, lse = api.paged_latent_decode_run(plan, q, pages, table)
    plan.check()
    ref = ref_decode(q, pages, table, [n], [0, 1], dl, math.log(2), False, 1.0, torch.float32)
    assert_close(out, lse, ref, rows[:, :dl].double().abs().sum(0) * 2.0 ** -32)


@pytest.mark.parametrize("at", [0, 10000, 19999])
@pytest.mark.parametrize("num_sms", [1, 152])
def test_prefill_small_weights(num_sms, at):
    n, lq, H = 20000, 5, 2
    g = torch.Generator(device=DEV).manual_seed(at)
    kv = torch.zeros((n, H, 256), dtype=HF, device=DEV)
    kv[..., 128:] = 0.5 + 0.5 * torch.rand((n, H, 128), generator=g, device=DEV)
    kv[at, :, 128:192] = 0
    rope = torch.zeros((n, 64), dtype=HF, device=DEV)
    rope[:, 0] = exponents(n, at, g)
    q = torch.zeros((lq, H, 192), dtype=HF, device=DEV)
    q[..., 128] = 1
    plan = api.batch_latent_prefill_plan([0, lq], [0, n], num_heads=H, causal=False, dtype=HF,
                                         sm_scale=math.log(2), out_dtype=torch.float32,
                                         return_lse=True, num_sms=num_sms)
    out, lse = api.batch_latent_prefill_run(plan, q, kv[..., :128], rope, kv[..., 128:])
    plan.check()
    _, ref = ref_prefill(q, kv[..., :128], rope, kv[..., 128:], [0, lq], [0, n], math.log(2), False,
                         1.0, torch.float32)
    assert_close(out, lse, ref, kv[..., 128:].double().abs().sum(0) * 2.0 ** -32)
