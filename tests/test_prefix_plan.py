"""The plan of decode behind shared prefixes (host only)."""

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api


def plan(lens, groups, pages, **kw):
    a = dict(num_qo_heads=8, num_kv_heads=2, page_size=16, max_pages_per_seq=4096, num_pages=10000, num_sms=152,
             host_only=True)
    a.update(kw)
    return api.paged_prefix_decode_plan(lens, groups, pages, **a)


@pytest.mark.parametrize("kw,code", [
    (dict(groups=[1, 4]), L.PKA_ERR_INVALID_ARG),
    (dict(groups=[0, 3]), L.PKA_ERR_INVALID_ARG),
    (dict(groups=[0, 5]), L.PKA_ERR_INVALID_ARG),
    (dict(groups=[0, 3, 2, 4], pages=[1, 1, 1]), L.PKA_ERR_INVALID_ARG),
    (dict(pages=[-1]), L.PKA_ERR_INVALID_ARG),
    (dict(pages=[11]), L.PKA_ERR_INVALID_ARG),                        # 176 keys, a request has 170
    (dict(pages=[10], causal=True, q_len=12), L.PKA_ERR_INVALID_ARG),   # its first row sees 159
    (dict(lens=[0, 200, 200, 200], pages=[0]), L.PKA_ERR_INVALID_ARG),
    (dict(page_size=24), L.PKA_ERR_UNSUPPORTED),
    (dict(head_dim=64), L.PKA_ERR_UNSUPPORTED),
    (dict(num_qo_heads=7), L.PKA_ERR_INVALID_ARG),
])
def test_refusals(kw, code):
    a = dict(lens=[170, 200, 200, 200], groups=[0, 4], pages=[4])
    a.update(kw)
    with pytest.raises(L.PkaError) as e:
        plan(**a)
    assert e.value.code == code


def test_refuses_a_window():
    d = L.DecodeDesc(batch_size=2, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, max_pages_per_seq=9,
                     num_pages=50, q_len=1, window_left=5, scale=1.0, bmm2_scale=1.0, num_sms=8,
                     flags=L.PKA_PLAN_HOST_ONLY)
    import ctypes
    i32 = lambda *x: (ctypes.c_int32 * len(x))(*x)   # noqa: E731
    h, ws = ctypes.c_void_p(), ctypes.c_size_t()
    rc = L.lib().paged_prefix_decode_plan(ctypes.byref(h), ctypes.byref(d), i32(100, 100), None, i32(0, 2), 1, i32(3),
                                          ctypes.byref(ws), None)
    assert rc == L.PKA_ERR_UNSUPPORTED and not h.value


def test_binding_refuses():
    with pytest.raises(ValueError, match="one entry more"):
        plan([100, 100], [0, 2], [1, 1])
    with pytest.raises(ValueError, match="one entry more"):
        plan([100, 100], [0, 2], [1], qo_indptr=[0, 1])
    p = plan([1600] * 4, [0, 4], [90])
    with pytest.raises(ValueError, match="not made by"):
        api.paged_prefix_decode_run(api.paged_decode_plan([100], num_qo_heads=8, num_kv_heads=2, page_size=16,
                                                          max_pages_per_seq=9, num_pages=50, num_sms=8,
                                                          host_only=True), *[torch.zeros(1)] * 4)
    assert not hasattr(p, "handle")   # no other entry point takes it for its own plan


def test_groups_without_anything_to_share_are_plain_decode():
    for lens, groups, pages in (([500, 600], [0, 2], [0]), ([500, 600], [0, 1, 2], [9, 9]), ([500], [0, 0, 1], [3, 9])):
        i = plan(lens, groups, pages).info
        plain = api.paged_decode_plan(lens, num_qo_heads=8, num_kv_heads=2, page_size=16, max_pages_per_seq=4096,
                                      num_pages=10000, num_sms=152, host_only=True).info
        assert i.pop("num_pieces") == 0 and set(i.pop("prefix_chunks")) == {0}
        assert i == plain


def test_pieces_and_states():
    """Pieces: every chunk of a group for each KV head and 256 rows; a request's states are its
    group's chunks and its own."""
    lens = [16384 + 40] * 80 + [4000 + i for i in range(70)] + [900]
    p = plan(lens, [0, 80, 150, 151], [1024, 200, 50], num_qo_heads=32, num_kv_heads=8)
    i = p.info
    a, b = i["prefix_chunks"][0], i["prefix_chunks"][80]
    assert i["prefix_chunks"] == [a] * 80 + [b] * 70 + [0]
    assert a > b >= 1
    # 80 requests of 4 rows: two tiles of 256; 70: two
    assert i["num_pieces"] == 8 * 2 * (a + b)
    assert i["total_q"] == 151 and i["kernel"] == L.PKA_KERNEL_MMA
    assert i["workspace_bytes"] >= i["partial_rows"] * 129 * 4
    assert i["partial_rows"] >= 32 * (80 * (a + 1) + 70 * (b + 1))


def test_update_keeps_the_plan_where_it_refuses():
    p = plan([3000] * 8, [0, 8], [100])
    before = p.info
    with pytest.raises(L.PkaError):
        p.update([3000] * 8, [0, 8], [190])
    with pytest.raises(L.PkaError):
        p.update([3000] * 8, [0, 7], [100])
    assert p.info == before and p.batch_size == 8
    p.update([2000] * 3 + [5000] * 6, [0, 3, 9], [50, 300], qo_indptr=[0, 1, 2, 5, 6, 7, 8, 9, 10, 11])
    assert p.batch_size == 9 and p.total_q == 11 and p.info["num_pieces"] > 0
