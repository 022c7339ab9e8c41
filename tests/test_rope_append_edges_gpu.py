"""Rotated appends of shapes at the ends of the range, through the Python entry point."""

import pytest
import torch

from paged_kv_attention_32_gb300 import api
from tests import pages_ref as ref
from tests.test_rope_append_gpu import case, close, pool_after

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("axes", [0, 1, 3])
def test_no_tokens(axes, fused):
    """A step without tokens writes nothing, rotated or not, and returns queries of no rows."""
    q, k, v, slots, pos, freq, (kp, vp) = case(0, 6, 2, 16, 128, (16, 24, 24)[:max(1, axes)], torch.bfloat16, 50,
                                               fused=fused)
    kept = kp.clone(), vp.clone()
    kw = dict(positions=pos if axes > 1 else pos[0], inv_freq=freq,
              sections=(16, 24, 24) if axes > 1 else None) if axes else {}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert api.paged_rope_append(k, v, slots, kp, vp, status=st, **kw) is None
    assert api.paged_rope_append(k, v, slots, kp, vp, q=q, status=st, **kw).shape == (0, 6, 128)
    assert api.paged_rope_append(k, v, slots, kp, vp, q=q, q_out=q, **kw) is q
    api.check_status(st)
    assert torch.equal(kp, kept[0]) and torch.equal(vp, kept[1])


@pytest.mark.parametrize("T", [1, 40])
def test_one_row_of_positions_for_all_axes(T):
    """Text among images: every axis has the token's place, one row expanded."""
    q, k, v, slots, pos, freq, (kp, vp) = case(T, 4, 2, 16, 128, (16, 24, 24), torch.bfloat16, 5000)
    same = pos[:1].expand(3, T)
    want_k = pool_after(kp, ref.rotate(k, same, freq, (16, 24, 24), "halves"), slots)
    out = api.paged_rope_append(k, v, slots, kp, vp, q=q, positions=same, inv_freq=freq, sections=(16, 24, 24))
    close(out, ref.rotate(q, same, freq, (16, 24, 24), "halves"), torch.bfloat16)
    close(kp, want_k, torch.bfloat16)


def restrided(x, at, stride):
    """x with another stride in a dimension of size 1, where it says nothing."""
    assert x.shape[at] == 1 and x.is_contiguous()
    s = list(x.stride())
    s[at] = stride
    y = x.as_strided(x.shape, s)
    assert y.is_contiguous() and y.contiguous().stride() == y.stride()
    return y


@pytest.mark.parametrize("odd", ["k", "v", "q", "q_out", "k_pages", "v_pages"])
@pytest.mark.parametrize("T,Hq,Hkv,pages,at", [(1, 4, 2, 3, 0), (5, 4, 1, 3, 1), (5, 1, 1, 1, 1), (1, 1, 1, 1, 0)])
def test_strides_of_dimensions_of_size_one(odd, T, Hq, Hkv, pages, at):
    """A single token's v as a slice of a fused projection is contiguous to torch whatever its stride, and
    k, normalised in between, has another: neither stride is used."""
    q, k, v, slots, pos, freq, _ = case(T, Hq, Hkv, 16, 128, (64,), torch.bfloat16, 500)
    t = dict(k=k.contiguous(), v=v.contiguous(), q=q.contiguous(), q_out=torch.empty_like(q.contiguous()))
    t = {n: x.clone(memory_format=torch.contiguous_format).view(-1).view(x.shape) for n, x in t.items()}
    t |= {n: torch.zeros((pages, Hkv, 16, 128), dtype=torch.bfloat16, device="cuda") for n in ("k_pages", "v_pages")}
    if t[odd].shape[at] == 1:
        t[odd] = restrided(t[odd], at, 1032 if odd.endswith("pages") else 12)
    slots = torch.randperm(pages * 16, device="cuda")[:T]
    want_k = pool_after(t["k_pages"], ref.rotate(k, pos, freq, (64,), "halves"), slots)
    want_v = pool_after(t["v_pages"], v.double(), slots)
    out = api.paged_rope_append(t["k"], t["v"], slots, t["k_pages"], t["v_pages"], q=t["q"], q_out=t["q_out"],
                                positions=pos, inv_freq=freq)
    close(out, ref.rotate(q, pos, freq, (64,), "halves"), torch.bfloat16)
    close(t["k_pages"], want_k, torch.bfloat16)
    assert torch.equal(t["v_pages"].double(), want_v)
    again = t["q"].clone()
    view = restrided(again, at, 8) if again.shape[at] == 1 else again   # the same rows: in place
    api.paged_rope_append(t["k"], t["v"], slots, t["k_pages"], t["v_pages"], q=again, q_out=view, positions=pos,
                          inv_freq=freq)
    assert torch.equal(again, out)


def test_prefix_decode_of_one_head_with_strides_that_say_nothing():
    from tests.test_prefix_gpu import check, make
    c = make([(9, [40, 3, 17])], heads=1, kv_heads=1, ps=16)
    want = check(c)
    c["v"], c["q"] = restrided(c["v"], 1, 24), restrided(c["q"], 1, 12)
    got = check(c)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
