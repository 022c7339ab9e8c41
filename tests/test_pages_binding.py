"""What the page operations and the rotated append refuse on the host (no GPU needed)."""

import ctypes

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api

P = 4096   # an aligned address that no refused call reads


def fork(**kw):
    a = dict(parents=P, children=P + 64, n=2, kv=P + 128, batch=4, free=P + 256, num_free=8, head=P + 320, ps=16,
             tables=P + 512, row=4, width=4, seq=P + 1024, src=P + 1152, dst=P + 1216, out=P + 1280, status=None)
    a.update(kw)
    return L.lib().paged_kv_fork(*a.values(), None)


def free(**kw):
    a = dict(rows=P, n=2, kv=P + 128, batch=4, free=P + 256, num_free=8, head=P + 320, ps=16, tables=P + 512, row=4,
             width=4, pages=100, seq=P + 1024, out=P + 1280, status=None)
    a.update(kw)
    return L.lib().paged_kv_free(*a.values(), None)


def compact(**kw):
    a = dict(kv=P + 128, batch=4, free=P + 256, num_free=8, head=P + 320, ps=16, tables=P + 512, row=4, width=4,
             pages=100, tables_out=P + 2048, out_row=4, free_out=P + 3328, src=P + 1152, dst=P + 1216, moves=8,
             count=P + 1280, status=None)
    a.update(kw)
    return L.lib().paged_kv_compact(*a.values(), None)


@pytest.mark.parametrize("call", [fork, free, compact])
@pytest.mark.parametrize("kw,code", [
    (dict(kv=None), L.PKA_ERR_INVALID_ARG),
    (dict(head=None), L.PKA_ERR_INVALID_ARG),
    (dict(tables=None), L.PKA_ERR_INVALID_ARG),
    (dict(batch=0), L.PKA_ERR_INVALID_ARG),
    (dict(batch=16385), L.PKA_ERR_UNSUPPORTED),
    (dict(num_free=-1), L.PKA_ERR_INVALID_ARG),
    (dict(free=None), L.PKA_ERR_INVALID_ARG),
    (dict(ps=0), L.PKA_ERR_INVALID_ARG),
    (dict(ps=65537), L.PKA_ERR_INVALID_ARG),
    (dict(width=0), L.PKA_ERR_INVALID_ARG),
    (dict(row=3), L.PKA_ERR_INVALID_ARG),
    (dict(kv=P + 130), L.PKA_ERR_INVALID_ARG),
])
def test_page_operations_refuse(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("call,kw,code", [
    (fork, dict(n=-1), L.PKA_ERR_INVALID_ARG),
    (fork, dict(n=5), L.PKA_ERR_INVALID_ARG),
    (fork, dict(src=None), L.PKA_ERR_INVALID_ARG),
    (fork, dict(seq=P + 128), L.PKA_ERR_INVALID_ARG),       # over kv_lens
    (fork, dict(out=P + 320), L.PKA_ERR_INVALID_ARG),       # over free_head
    (fork, dict(dst=P + 1152), L.PKA_ERR_INVALID_ARG),      # both moves
    (fork, dict(status=P + 1028), L.PKA_ERR_INVALID_ARG),   # inside seq_lens
    (free, dict(n=5), L.PKA_ERR_INVALID_ARG),
    (free, dict(rows=None), L.PKA_ERR_INVALID_ARG),
    (free, dict(pages=0), L.PKA_ERR_INVALID_ARG),
    (free, dict(pages=(1 << 22) + 1), L.PKA_ERR_UNSUPPORTED),
    (free, dict(seq=P + 128), L.PKA_ERR_INVALID_ARG),
    (free, dict(free=P + 512), L.PKA_ERR_INVALID_ARG),      # the list over the tables
    (compact, dict(pages=(1 << 22) + 1), L.PKA_ERR_UNSUPPORTED),
    (compact, dict(out_row=3), L.PKA_ERR_INVALID_ARG),
    (compact, dict(free_out=None), L.PKA_ERR_INVALID_ARG),
    (compact, dict(moves=-1), L.PKA_ERR_INVALID_ARG),
    (compact, dict(dst=None), L.PKA_ERR_INVALID_ARG),
    (compact, dict(tables_out=P + 516), L.PKA_ERR_INVALID_ARG),              # the tables, shifted
    (compact, dict(tables_out=P + 512, out_row=5), L.PKA_ERR_INVALID_ARG),   # or laid out otherwise
    (compact, dict(free_out=P + 260), L.PKA_ERR_INVALID_ARG),
])
def test_one_operation_refuses(call, kw, code):
    assert call(**kw) == code


def copy(pools=(P,), strides=(64,), sizes=(64,), pages=10, src=P + 1024, dst=P + 2048, n=4, count=None, status=None):
    m = len(pools)
    return L.lib().paged_kv_copy((ctypes.c_void_p * m)(*pools), (ctypes.c_int64 * m)(*strides),
                                 (ctypes.c_int64 * m)(*sizes), m, pages, src, dst, n, count, status, None)


@pytest.mark.parametrize("kw", [
    dict(pools=(P + 8,)), dict(pools=(None,)), dict(strides=(72,)), dict(sizes=(72,), strides=(80,)),
    dict(strides=(48,)), dict(pages=0), dict(pages=2 ** 31), dict(src=None), dict(n=-1), dict(count=P + 2),
    dict(strides=(2 ** 62,)), dict(pools=(P, P + 4096 + 4), strides=(64, 64), sizes=(64, 64)),
])
def test_copy_refuses(kw):
    assert copy(**kw) == L.PKA_ERR_INVALID_ARG


def rope(**kw):
    a = dict(q=P, q_tok=512, q_head=128, q_out=P + 65536, o_tok=512, o_head=128, Hq=4, k=P + 131072, v=P + 196608,
             kv_tok=256, kv_head=128, Hkv=2, D=128, pos=P, pos_row=8, freq=P, rotary=128, axes=2,
             sections=(ctypes.c_int32 * 4)(30, 34, 0, 0), pairs=0, slots=P, T=8, kp=P + 262144, vp=P + 524288,
             pages=10, ps=16, page=4096, head=2048, dtype=0, status=None)
    a.update(kw)
    return L.lib().paged_rope_append(*a.values(), None)


def sections(*x):
    return (ctypes.c_int32 * 4)(*x)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), L.PKA_ERR_UNSUPPORTED),
    (dict(D=64), L.PKA_ERR_UNSUPPORTED),
    (dict(T=-1), L.PKA_ERR_INVALID_ARG),
    (dict(T=2 ** 31), L.PKA_ERR_INVALID_ARG),
    (dict(Hkv=0), L.PKA_ERR_INVALID_ARG),
    (dict(q=None), L.PKA_ERR_INVALID_ARG),
    (dict(q_out=None), L.PKA_ERR_INVALID_ARG),
    (dict(Hq=0), L.PKA_ERR_INVALID_ARG),
    (dict(k=None), L.PKA_ERR_INVALID_ARG),
    (dict(slots=None), L.PKA_ERR_INVALID_ARG),
    (dict(rotary=130), L.PKA_ERR_INVALID_ARG),
    (dict(rotary=24), L.PKA_ERR_INVALID_ARG),
    (dict(rotary=144), L.PKA_ERR_INVALID_ARG),
    (dict(pos=None), L.PKA_ERR_INVALID_ARG),
    (dict(freq=None), L.PKA_ERR_INVALID_ARG),
    (dict(freq=P + 4), L.PKA_ERR_INVALID_ARG),
    (dict(sections=None), L.PKA_ERR_INVALID_ARG),
    (dict(sections=sections(30, 33)), L.PKA_ERR_INVALID_ARG),
    (dict(sections=sections(-1, 65)), L.PKA_ERR_INVALID_ARG),
    (dict(sections=sections(2 ** 31 - 1, 2 ** 31 - 1)), L.PKA_ERR_INVALID_ARG),
    (dict(axes=0), L.PKA_ERR_INVALID_ARG),
    (dict(axes=5), L.PKA_ERR_INVALID_ARG),
    (dict(pairs=2), L.PKA_ERR_INVALID_ARG),
    (dict(pos_row=7), L.PKA_ERR_INVALID_ARG),
    (dict(q_tok=514), L.PKA_ERR_INVALID_ARG),
    (dict(kv_head=-128), L.PKA_ERR_INVALID_ARG),
    (dict(kp=P + 8), L.PKA_ERR_INVALID_ARG),
    (dict(slots=P + 4), L.PKA_ERR_INVALID_ARG),
    (dict(pages=0), L.PKA_ERR_INVALID_ARG),
    (dict(ps=0), L.PKA_ERR_INVALID_ARG),
    (dict(q_out=P + 1024), L.PKA_ERR_INVALID_ARG),            # over q without being q
    (dict(q_out=P, o_tok=1024), L.PKA_ERR_INVALID_ARG),
    (dict(q_out=P + 131072), L.PKA_ERR_INVALID_ARG),          # over k, over v
    (dict(q_out=P + 196608 + 512), L.PKA_ERR_INVALID_ARG),
    (dict(o_tok=0), L.PKA_ERR_INVALID_ARG),                   # rows written twice
    (dict(o_head=64), L.PKA_ERR_INVALID_ARG),
    (dict(q_out=P, o_tok=512, o_head=0, q_head=0), L.PKA_ERR_INVALID_ARG),
    (dict(head=1024), L.PKA_ERR_INVALID_ARG),
    (dict(page=1024), L.PKA_ERR_INVALID_ARG),
    (dict(vp=P + 262144), L.PKA_ERR_INVALID_ARG),             # keys and values to one pool
])
def test_rope_append_refuses(kw, code):
    assert rope(**kw) == code


def test_rope_append_of_no_tokens_runs_nothing():
    assert rope(T=0) == L.PKA_OK
    assert rope(T=0, k=None, v=None, slots=None, kp=None, vp=None) == L.PKA_OK


def test_pools_of_a_copy():
    a = torch.zeros((4, 2, 16))
    with pytest.raises(ValueError, match="at least one"):
        api.KvPools([])
    with pytest.raises(ValueError, match="same number of pages"):
        api.KvPools([a, torch.zeros((5, 16))])
    with pytest.raises(ValueError, match="dense"):
        api.KvPools([a[:, :, ::2]])
    pools = api.KvPools([torch.zeros((4, 2, 2, 16))[:, 1], a])
    assert list(pools.c[1]) == [256, 128] and list(pools.c[2]) == [128, 128]
