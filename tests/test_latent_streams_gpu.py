"""Latent entry points on a stream that is not the current one: what they read is written there
by work that is still running when they are called."""
import pytest
import torch

from latent_ref import assert_within, ref_decode
from paged_kv_attention_32_gb300 import api

pytestmark = pytest.mark.gpu

DEV, BF = "cuda", torch.bfloat16
BUSY = 50_000_000   # cycles, some 25 ms


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _side(raw):
    s = torch.cuda.Stream()
    return s, (s.cuda_stream if raw else s)


@pytest.mark.parametrize("raw", [False, True])
def test_append_waits_for_the_slots_of_its_own_stream(raw):
    rows = torch.randn((40, 320), device=DEV).to(BF)
    pages = torch.zeros((6, 16, 320), dtype=BF, device=DEV)
    made = torch.randperm(96, device=DEV)[:40]
    slots = torch.full((40,), -1, dtype=torch.int64, device=DEV)
    want = pages.clone()
    want.view(96, 320)[made] = rows
    torch.cuda.synchronize()
    side, stream = _side(raw)
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        slots.copy_(made)
    api.paged_latent_append(rows[:, :256], rows[:, 256:], slots, pages, stream=stream)
    side.synchronize()
    assert torch.equal(pages, want)


@pytest.mark.parametrize("raw", [False, True])
def test_a_step_on_one_given_stream(raw):
    """Tables, append and decode, each given the stream: every one reads what the last wrote."""
    B, H, dl, ps, D = 3, 16, 256, 16, 320
    new = [37, 1, 64]
    rows = torch.randn((102, D), device=DEV).to(BF)
    q = torch.randn((B, H, D), device=DEV).to(BF)
    free, table = torch.arange(20, dtype=torch.int32, device=DEV).flip(0), i32([[-1] * 8] * B)
    pages = torch.full((20, ps, D), float("nan"), dtype=BF, device=DEV)
    plan = api.paged_latent_decode_plan([8 * ps] * B, num_heads=H, page_size=ps, scale=0.06,
                                        max_pages_per_seq=8, num_pages=20, latent_dim=dl,
                                        return_lse=True, freeze_seq_lens=False)
    lens, head, status, new_dev = i32([0] * B), i32([0]), i32([0]), i32([0] * B)
    made = i32(new)
    torch.cuda.synchronize()
    side, stream = _side(raw)
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        new_dev.copy_(made)
    t = api.paged_kv_tables(lens, new_dev, free, head, table, page_size=ps, num_slots=102,
                            status=status, stream=stream)
    api.paged_latent_append(rows[:, :dl], rows[:, dl:], t.slot_map, pages, status=status,
                            stream=stream)
    out, lse = api.paged_latent_decode_run(plan, q, pages, table, seq_lens_kv=t.seq_lens,
                                           stream=stream)
    side.synchronize()
    api.check_status(status, stream=stream)
    plan.check(stream=stream)
    assert t.seq_lens.tolist() == new
    dense = torch.zeros((B, 8 * ps, D), dtype=BF, device=DEV)
    at = 0
    for b, n in enumerate(new):
        dense[b, :n] = rows[at:at + n]
        at += n
    ids = torch.arange(B * 8, device=DEV).view(B, 8)
    assert_within(out, lse, ref_decode(q, dense.view(-1, ps, D), ids, new, list(range(B + 1)), dl,
                                       0.06, False, 1.0, BF))


def test_handle_0_is_the_default_stream():
    """The raw handle that torch gives for its default stream, from under another stream."""
    rows = torch.randn((40, 320), device=DEV).to(BF)
    pages = torch.zeros((6, 16, 320), dtype=BF, device=DEV)
    lens, new, made = i32([0]), i32([0]), i32([40])
    free, head, table = torch.arange(6, dtype=torch.int32, device=DEV), i32([0]), i32([[-1] * 6])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle = torch.cuda.default_stream().cuda_stream
    assert handle == 0
    torch.cuda._sleep(BUSY)
    new.copy_(made)
    with torch.cuda.stream(side):
        t = api.paged_kv_tables(lens, new, free, head, table, page_size=16, num_slots=40, stream=handle)
        api.paged_latent_append(rows[:, :256], rows[:, 256:], t.slot_map, pages, stream=handle)
    torch.cuda.default_stream().synchronize()
    assert torch.equal(pages.view(96, 320)[:40], rows) and t.seq_lens.tolist() == [40]
