"""Latent entry points at the edges of what they take."""
import pytest
import torch

from latent_ref import assert_within, ref_decode
from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api

pytestmark = pytest.mark.gpu

DEV, BF = "cuda", torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_table_rows_over_one_another_are_refused_and_one_row_is_not():
    """Requests that share one row of pages by a row stride of 0; of one request the stride
    says nothing."""
    q = torch.randn((3, 8, 320), device=DEV).to(BF)
    pages = torch.randn((6, 16, 320), device=DEV).to(BF)
    room = torch.full((16,), 10 ** 6, dtype=torch.int32, device=DEV)
    room[:4] = i32([5, 1, 3, 0])
    before = room.clone()
    args = dict(num_heads=8, page_size=16, max_pages_per_seq=4, num_pages=6, scale=0.05,
                latent_dim=256, return_lse=True)
    plan = api.paged_latent_decode_plan([50] * 3, **args)
    for rows in (room[:4].expand(3, 4), room.as_strided((3, 4), (2, 1))):
        with pytest.raises(L.PkaError, match="bt_row_stride") as e:
            api.paged_latent_decode_run(plan, q, pages, rows)
        assert e.value.code == L.PKA_ERR_INVALID_ARG
        with pytest.raises(L.PkaError, match="row stride"):
            api.paged_kv_tables(i32([0] * 3), i32([1] * 3), i32([0, 1, 2]), i32([0]), rows,
                                page_size=16, num_slots=3)
    torch.cuda.synchronize()
    assert torch.equal(room, before)
    one = api.paged_latent_decode_plan([50], **args)
    for stride in (0, 1, 4, 12):
        table = room.as_strided((1, 4), (stride, 1))
        out, lse = api.paged_latent_decode_run(one, q[:1], pages, table)
        one.check()
        assert_within(out, lse, ref_decode(q[:1], pages, table, [50], [0, 1], 256, 0.05, False, 1.0, BF))


def test_decode_of_a_batch_without_query_rows():
    """Every request idle: nothing is written, an empty q (and its null address) is fine."""
    pages = torch.randn((6, 16, 320), device=DEV).to(BF)
    table, q = i32([[5, 1, 3, 0]] * 3), torch.randn((3, 8, 320), device=DEV).to(BF)
    args = dict(num_heads=8, page_size=16, max_pages_per_seq=4, num_pages=6, scale=0.05,
                latent_dim=256, return_lse=True)
    plan = api.paged_latent_decode_plan([50, 0, 3], qo_indptr=[0, 0, 0, 0], **args)
    assert plan.total_q == 0
    out, lse = api.paged_latent_decode_run(plan, q[:0], pages, table)
    assert out.shape == (0, 8, 256) and lse.shape == (0, 8)
    kept, kept_lse = torch.full((3, 8, 256), 7.0, dtype=BF, device=DEV), torch.full((3, 8), 7.0, device=DEV)
    api.paged_latent_decode_run(plan, q, pages, table, out=kept, lse=kept_lse)
    plan.check()
    assert bool((kept == 7).all()) and bool((kept_lse == 7).all())
    # from idle to rows and back, by update
    plan.update([50, 17, 3], qo_indptr=[0, 1, 2, 3])
    out, lse = api.paged_latent_decode_run(plan, q, pages, table)
    plan.check()
    assert_within(out, lse, ref_decode(q, pages, table, [50, 17, 3], [0, 1, 2, 3], 256, 0.05, False,
                                       1.0, BF))
    plan.update([50, 17, 3], qo_indptr=[0, 0, 0, 0])
    out, _ = api.paged_latent_decode_run(plan, q[:0], pages, table)
    plan.check()
    assert out.shape == (0, 8, 256)
    with pytest.raises(L.PkaError, match="NULL"):
        L.check(L.lib().paged_latent_decode_run(None, None, 0, 0, None, 0, None, 0, None, None, None,
                                                None, 0, None), "run")


@pytest.mark.parametrize("lk", [[0, 0], [0, 70]])
def test_prefill_of_a_batch_without_query_rows(lk):
    ko = [0, lk[0], lk[0] + lk[1]]
    q = torch.randn((2, 3, 192), device=DEV).to(BF)
    kv, rope = torch.randn((ko[-1], 3, 256), device=DEV).to(BF), torch.randn((ko[-1], 64), device=DEV).to(BF)
    plan = api.batch_latent_prefill_plan([0, 0, 0], ko, num_heads=3, return_lse=True)
    run = api.batch_latent_prefill_run
    out, lse = run(plan, q[:0], kv[..., :128], rope, kv[..., 128:])
    assert out.shape == (0, 3, 128) and lse.shape == (0, 3)
    kept, kept_lse = torch.full((2, 3, 128), 7.0, dtype=BF, device=DEV), torch.full((2, 3), 7.0, device=DEV)
    run(plan, q, kv[..., :128], rope, kv[..., 128:], out=kept, lse=kept_lse)
    plan.check()
    assert bool((kept == 7).all()) and bool((kept_lse == 7).all())
