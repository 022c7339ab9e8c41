"""Rotated keys and values in the paged pools against the rotation in 64 bits."""

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api
from tests import pages_ref as ref

pytestmark = pytest.mark.gpu

D = 128


def close(got, want, dtype):
    """One rounding to ``dtype`` (half a step of the value) and the 32-bit rotation before it:
    two products and a sum of values of at most |x0| + |x1|, with cos and sin of an angle that
    is off by half a step of a turn fraction (2^-25 turns: 2e-7) and themselves by 2^-23, all
    below 2^-20 of the largest value; steps below the type's smallest normal number count as it."""
    eps = torch.finfo(dtype).eps / 2
    bound = eps * want.abs() + 2.0 ** -20 * want.abs().max() + torch.finfo(dtype).smallest_normal * eps
    bad = (got.double() - want).abs() > bound
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}"


def case(T, Hq, Hkv, ps, rotary, sections, dtype, far, seed=0, extra=3, fused=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.Generator().manual_seed(seed)
    if fused:
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dtype)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:   # heads outermost
        q = torch.randn((Hq, T, D), generator=g, device="cuda").to(dtype).transpose(0, 1)
        kv = torch.randn((2, Hkv, T, D), generator=g, device="cuda").to(dtype)
        k, v = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    pages = -(-T // ps) + extra
    slots = torch.randperm(pages * ps, generator=c)[:T].cuda()
    pos = torch.randint(-3, far, (len(sections), T), generator=c, dtype=torch.int64).to(torch.int32).cuda()
    freq = 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) / max(1, rotary // 2))
    pools = [torch.randn((pages, Hkv, ps, D), generator=g, device="cuda").to(dtype) for _ in range(2)]
    return q, k, v, slots, pos, freq.cuda(), pools


def pool_after(pool, rows, slots):
    ps = pool.shape[2]
    want = pool.double().clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pool.shape[0] * ps:
            want[s // ps, :, s % ps] = rows[t]
    return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("T,Hq,Hkv,ps,rotary,sections,far", [
    (1, 1, 1, 16, 128, (64,), 131072),
    (3, 5, 1, 48, 64, (32,), 10),
    (64, 32, 8, 16, 128, (16, 24, 24), 5000),
    (607, 4, 2, 16, 96, (0, 48), 1000),
    (609, 7, 3, 64, 32, (4, 4, 4, 4), 2 ** 31 - 1),
    (1001, 16, 2, 32, 16, (3, 5), 500000),
])
def test_rope_append(dtype, pairs, T, Hq, Hkv, ps, rotary, sections, far):
    q, k, v, slots, pos, freq, (kp, vp) = case(T, Hq, Hkv, ps, rotary, sections, dtype, far, fused=T % 2 == 1)
    want_q = ref.rotate(q, pos, freq, sections, pairs)
    want_k = pool_after(kp, ref.rotate(k, pos, freq, sections, pairs), slots)
    want_v = pool_after(vp, v.double(), slots)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_rope_append(k, v, slots, kp, vp, q=q, positions=pos, inv_freq=freq, sections=sections,
                                pairs=pairs, status=st)
    api.check_status(st)
    close(out, want_q, dtype)
    close(kp, want_k, dtype)
    assert torch.equal(vp.double(), want_v)


@pytest.mark.parametrize("T", [1, 5, 640])
def test_without_rotation_and_without_queries(T):
    q, k, v, slots, pos, freq, (kp, vp) = case(T, 4, 2, 16, 128, (64,), torch.bfloat16, 100)
    want_k, want_v = pool_after(kp, k.double(), slots), pool_after(vp, v.double(), slots)
    assert api.paged_rope_append(k, v, slots, kp, vp) is None
    assert torch.equal(kp.double(), want_k) and torch.equal(vp.double(), want_v)
    out = api.paged_rope_append(k, v, slots, kp, vp, q=q)
    assert torch.equal(out, q)
    assert api.paged_rope_append(k, v, slots, kp, vp, positions=pos[0], inv_freq=freq) is None
    close(kp, pool_after(kp, ref.rotate(k, pos, freq, (64,), "halves"), slots), torch.bfloat16)


@pytest.mark.parametrize("T", [9, 700])
def test_queries_in_place_of_a_fused_projection(T):
    q, k, v, slots, pos, freq, (kp, vp) = case(T, 6, 2, 16, 64, (32,), torch.float16, 9000)
    want, kept_k, kept_v = ref.rotate(q, pos, freq, (32,), "neighbours"), k.clone(), v.clone()
    out = api.paged_rope_append(k, v, slots, kp, vp, q=q, q_out=q, positions=pos, inv_freq=freq, pairs="neighbours")
    assert out is q
    close(q, want, torch.float16)
    assert torch.equal(k, kept_k) and torch.equal(v, kept_v)


def test_skipped_slots_and_slots_past_the_pool():
    q, k, v, slots, pos, freq, (kp, vp) = case(10, 2, 2, 16, 128, (64,), torch.bfloat16, 50)
    slots[2], slots[7] = -1, -(2 ** 40)
    slots[4] = kp.shape[0] * 16
    slots[9] = 2 ** 62
    rows = ref.rotate(k, pos, freq, (64,), "halves")
    want_k, want_v = pool_after(kp, rows, slots), pool_after(vp, v.double(), slots)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_rope_append(k, v, slots, kp, vp, q=q, positions=pos, inv_freq=freq, status=st)
    with pytest.raises(L.PkaError) as e:
        api.check_status(st)
    assert e.value.code == L.PKA_ERR_DEVICE_BOUNDS
    api.check_status(st)   # read and cleared
    close(out, ref.rotate(q, pos, freq, (64,), "halves"), torch.bfloat16)
    close(kp, want_k, torch.bfloat16)
    assert torch.equal(vp.double(), want_v)


def test_infinities_and_nan_stay_in_their_pairs():
    q, k, v, slots, pos, freq, (kp, vp) = case(4, 2, 1, 16, 64, (32,), torch.bfloat16, 50)
    k[1, 0, 3] = float("nan")
    k[2, 0, 100] = float("inf")
    v[0, 0, 5] = float("nan")
    api.paged_rope_append(k, v, slots, kp, vp, positions=pos, inv_freq=freq)
    flat_k, flat_v = kp.transpose(1, 2).reshape(-1, 1, D)[slots], vp.transpose(1, 2).reshape(-1, 1, D)[slots]
    assert flat_k[1, 0].isnan().nonzero().flatten().tolist() == [3, 35]
    assert flat_k[2, 0].isinf().nonzero().flatten().tolist() == [100]
    assert flat_v[0, 0].isnan().nonzero().flatten().tolist() == [5]


def test_offsets_past_32_bits_in_a_combined_pool():
    """K and V halves of one tensor of 2.5e9 values."""
    pages, ps = 300000, 16
    both = torch.zeros((pages, 2, 2, ps, D), dtype=torch.bfloat16, device="cuda")
    kp, vp = both[:, 0], both[:, 1]
    k = torch.ones((2, 2, D), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([pages * ps - 1, 3], device="cuda")
    api.paged_rope_append(k, 2 * k, slots, kp, vp)
    assert bool((both[-1, 0, :, -1] == 1).all()) and bool((both[-1, 1, :, -1] == 2).all())
    assert bool((both[0, 1, :, 3] == 2).all()) and int(torch.count_nonzero(both)) == 2 * 2 * 2 * D


def test_captured_and_replayed():
    q, k, v, slots, pos, freq, (kp, vp) = case(33, 4, 2, 16, 128, (20, 44), torch.bfloat16, 4000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        api.paged_rope_append(k, v, slots, kp, vp, q=q, positions=pos, inv_freq=freq, sections=(20, 44))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.paged_rope_append(k, v, slots, kp, vp, q=q, positions=pos, inv_freq=freq, sections=(20, 44))
    for add in (1, 100):
        pos += add
        graph.replay()
        close(out, ref.rotate(q, pos, freq, (20, 44), "halves"), torch.bfloat16)
        close(kp, pool_after(kp, ref.rotate(k, pos, freq, (20, 44), "halves"), slots), torch.bfloat16)
