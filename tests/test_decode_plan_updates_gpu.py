"""Updates that CUDA refuses, and the runs after them: plans behind shared prefixes that come to share
nothing, and ordinary decode plans."""

import ctypes

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api
from tests import prefix_ref as ref
from tests.test_prefix_gpu import check, close, make, plan_of, table

pytestmark = pytest.mark.gpu

N = 4096   # requests whose lists outgrow any buffer of a small plan


def refused(update):
    """An allocation is refused while a stream of this thread captures."""
    cudart = ctypes.CDLL("libcudart.so.13")
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), ctypes.c_void_p()
    assert cudart.cudaStreamBeginCapture(ctypes.c_void_p(s.cuda_stream), 1) == 0
    try:
        with pytest.raises(L.PkaError) as e:
            update(s)
    finally:
        cudart.cudaStreamEndCapture(ctypes.c_void_p(s.cuda_stream), ctypes.byref(graph))
        cudart.cudaGetLastError()
    assert e.value.code == L.PKA_ERR_CUDA


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("been", [False, True])
def test_prefix_plans_that_come_to_share_nothing(shared, been):
    c = make([(30, [40, 30, 300]), (5, [9, 9])], heads=8, kv_heads=2, ps=16, seed=1)
    to = lambda pre: p.update(c["kv"], c["groups"], pre, qo_indptr=c["qo"])   # noqa: E731
    p = plan_of(c if shared else c | {"pre": [0, 0]})
    if been:   # buffers of both kinds
        to([0, 0] if shared else c["pre"])
        to(c["pre"] if shared else [0, 0])
    check(c, plan=p, pieces=shared)
    info, ws = p.info, p.workspace_bytes
    refused(lambda s: p.update([480] * N, [0, N], [0], stream=s))
    assert p.info == info and p.workspace_bytes == ws
    check(c, plan=p, pieces=shared)
    to([0, 0])
    check(c, plan=p, pieces=False)
    to(c["pre"])
    check(c, plan=p)


def test_decode_plans():
    c = make([(0, [40, 900, 17, 300])], heads=8, kv_heads=2, ps=16, seed=2)
    p = api.paged_decode_plan(c["kv"], num_qo_heads=8, num_kv_heads=2, page_size=16, max_pages_per_seq=c["width"],
                              num_pages=c["k"].shape[0], scale=c["scale"], return_lse=True)
    want = ref.decode(c["q"], c["k"], c["v"], c["tables"], c["kv"], c["qo"], causal=False, scale=c["scale"])
    run = lambda: close(api.paged_decode_run(p, c["q"], c["k"], c["v"], table(c)), want, c["v"], c["dtype"], c["dtype"])   # noqa: E731
    run()
    info, ws = p.info, p.workspace_bytes
    refused(lambda s: p.update([480] * N, stream=s))
    assert p.info == info and p.workspace_bytes == ws
    run()
    p.update(c["kv"])
    run()
    p.check()
