"""What one CTA of a pair writes to shared memory and the other's tensor-core products read: the
weights of a tile, queries by plain loads, values cleared behind the last key."""
import pytest
import torch

from latent_ref import assert_within, ref_decode, ref_prefill
from paged_kv_attention_32_gb300 import api

pytestmark = pytest.mark.gpu

DEV, BF = "cuda", torch.bfloat16


@pytest.mark.parametrize("heads", [72, 100, 128])   # queries by copies, by plain loads, by copies
@pytest.mark.parametrize("dl", [256, 512])
def test_decode_pairs_hand_over_every_tile(heads, dl):
    """Scores spread so wide that a row's weights lie on other keys in every tile: a tile
    multiplied by an earlier one's weights, or by values not yet cleared, is far off.  Many
    pieces per pair, each with a last tile that is not full, over and over beside copies that
    keep the memory busy; the first run is checked in 64 bits, the others have its bits."""
    kv = [64 * (1 + b % 5) - 37 + b % 3 for b in range(40)]
    g = torch.Generator(device=DEV).manual_seed(heads + dl)
    need = [-(-n // 16) for n in kv]
    pages = torch.full((sum(need), 16, dl + 64), float("nan"), dtype=BF, device=DEV)
    table = torch.zeros((40, max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(kv):
        table[b, :need[b]] = torch.arange(at, at + need[b])
        rows = torch.full((need[b] * 16, dl + 64), float("nan"), dtype=BF, device=DEV)
        rows[:n] = torch.randn((n, dl + 64), generator=g, device=DEV).to(BF)
        pages[at:at + need[b]] = rows.view(-1, 16, dl + 64)
        at += need[b]
    table = table.to(DEV)
    q = torch.randn((40, heads, dl + 64), generator=g, device=DEV).to(BF)
    scale = 8 / (dl + 64) ** 0.5
    for sms in (2, 16, 152):
        plan = api.paged_latent_decode_plan(kv, num_heads=heads, page_size=16, scale=scale,
                                            max_pages_per_seq=table.shape[1], num_sms=sms,
                                            num_pages=pages.shape[0], latent_dim=dl, return_lse=True,
                                            out_dtype=torch.float32)
        first = api.paged_latent_decode_run(plan, q, pages, table)
        plan.check()
        assert_within(*first, ref_decode(q, pages, table, kv, list(range(41)), dl, scale, False, 1.0,
                                         torch.float32))
        big = torch.zeros(1 << 26, dtype=torch.int32, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for i in range(20):
                big.add_(i)
        for _ in range(40):
            out, lse = api.paged_latent_decode_run(plan, q, pages, table)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        plan.check()
        torch.cuda.synchronize()


@pytest.mark.parametrize("num_sms", [1, 20, 152])
def test_prefill_pairs_hand_over_cleared_values(num_sms):
    """Requests whose last key tile is followed by NaN, many of them for every pair, over and
    over; the first run is checked in 64 bits, the others have its bits."""
    g = torch.Generator(device=DEV).manual_seed(num_sms)
    lq, lk = [3, 1, 40, 2, 129, 1] * 6, [70, 1, 100, 129, 700, 63] * 6
    gap, H = 64, 3
    qo, ko = [0], [0]
    for a, b in zip(lq, lk):   # every request's keys, then a request of junk without queries
        qo += [qo[-1] + a] * 2
        ko += [ko[-1] + b, ko[-1] + b + gap]
    q = torch.randn((qo[-1], H, 192), generator=g, device=DEV).to(BF)
    kv = torch.randn((ko[-1], H, 256), generator=g, device=DEV).to(BF)
    rope = torch.randn((ko[-1], 64), generator=g, device=DEV).to(BF)
    for a, b in zip(ko[1::2], ko[2::2]):
        kv[a:b] = float("nan")
        rope[a:b] = float("nan")
    k, v = kv[..., :128], kv[..., 128:]
    plan = api.batch_latent_prefill_plan(qo, ko, num_heads=H, return_lse=True, num_sms=num_sms,
                                         out_dtype=torch.float32)
    first = api.batch_latent_prefill_run(plan, q, k, rope, v)
    plan.check()
    _, ref = ref_prefill(q, k, rope, v, qo, ko, 192 ** -0.5, True, 1.0, torch.float32)
    assert_within(*first, ref)
    for _ in range(40):
        out, lse = api.batch_latent_prefill_run(plan, q, k, rope, v)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    plan.check()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("past,num_sms,cut", [(900, 2, False), (900, 152, False), (3000, 152, True)])
def test_prefill_warps_of_which_some_lanes_store(past, num_sms, cut, out_dtype):
    """Every count of live rows in a warp, of whole tiles and of tiles cut along their keys;
    rows behind them left as they were."""
    lq = list(range(1, 34)) + [160, 129]
    lk = [n + past for n in lq]
    g = torch.Generator(device=DEV).manual_seed(2)
    qo, ko = [0], [0]
    for a, b in zip(lq, lk):
        qo.append(qo[-1] + a)
        ko.append(ko[-1] + b)
    q = torch.randn((qo[-1], 1, 192), generator=g, device=DEV).to(BF)
    kv = torch.randn((ko[-1], 1, 256), generator=g, device=DEV).to(BF)
    rope = torch.randn((ko[-1], 64), generator=g, device=DEV).to(BF)
    plan = api.batch_latent_prefill_plan(qo, ko, num_heads=1, return_lse=True, num_sms=num_sms,
                                         out_dtype=out_dtype)
    assert (plan.workspace_bytes > 0) == cut
    out = torch.full((qo[-1] + 7, 1, 128), 7.0, dtype=out_dtype, device=DEV)
    lse = torch.full((qo[-1] + 7, 1), 7.0, device=DEV)
    q = torch.cat([q, q[:7]])
    api.batch_latent_prefill_run(plan, q, kv[..., :128], rope, kv[..., 128:], out=out, lse=lse)
    plan.check()
    n = qo[-1]
    _, ref = ref_prefill(q[:n], kv[..., :128], rope, kv[..., 128:], qo, ko, 192 ** -0.5, True, 1.0,
                         out_dtype)
    assert_within(out[:n], lse[:n], ref)
    assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())


@pytest.mark.parametrize("heads", [1, 9, 15, 31, 47, 63, 65, 90, 97, 127])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_decode_warps_of_which_some_lanes_store(heads, out_dtype):
    kv, dl = [130, 5, 700, 64], 256
    g = torch.Generator(device=DEV).manual_seed(heads)
    pages = torch.randn((64, 16, dl + 64), generator=g, device=DEV).to(BF)
    table = torch.randperm(64, generator=torch.Generator().manual_seed(heads)).to(torch.int32)
    table = table.repeat(3).view(4, 48).to(DEV)
    q = torch.randn((6, heads, dl + 64), generator=g, device=DEV).to(BF)
    for sms in (4, 152):
        plan = api.paged_latent_decode_plan(kv, num_heads=heads, page_size=16, scale=0.05,
                                            max_pages_per_seq=48, num_pages=64, latent_dim=dl,
                                            return_lse=True, out_dtype=out_dtype, num_sms=sms)
        out = torch.full((6, heads, dl), 7.0, dtype=out_dtype, device=DEV)
        lse = torch.full((6, heads), 7.0, device=DEV)
        api.paged_latent_decode_run(plan, q, pages, table, out=out, lse=lse)
        plan.check()
        assert_within(out[:4], lse[:4], ref_decode(q, pages, table, kv, list(range(5)), dl, 0.05, False,
                                                   1.0, out_dtype))
        assert bool((out[4:] == 7).all()) and bool((lse[4:] == 7).all())
