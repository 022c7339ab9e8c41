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
