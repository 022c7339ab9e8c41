"""What the binding refuses of tensors on a device, before anything runs, and workspaces that calls
share."""

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from paged_kv_attention_32_gb300 import api
from tests import prefix_ref as ref
from tests.test_prefix_gpu import close, make, plan_of, table

pytestmark = pytest.mark.gpu

CASE = dict(groups=[(20, [40, 30, 35])], heads=8, kv_heads=2, ps=16)


def prefix_case():
    c = make(**CASE)
    p = plan_of(c)
    return p, dict(q=c["q"], k_pages=c["k"], v_pages=c["v"], block_tables=table(c)), c


@pytest.mark.parametrize("name,change", [
    ("q", lambda x: x.float()), ("q", lambda x: x.half()), ("q", lambda x: x.cpu()), ("q", lambda x: x[:2]),
    ("q", lambda x: x[:, :4]), ("q", lambda x: x[:, 0]), ("q", lambda x: x.transpose(1, 2)),
    ("k_pages", lambda x: x[:-1]), ("k_pages", lambda x: x.half()), ("k_pages", lambda x: x.cpu()),
    ("v_pages", lambda x: x[:, :1]), ("v_pages", lambda x: torch.stack([x, x], 1)[:, 0]),
    ("block_tables", lambda x: x.long()), ("block_tables", lambda x: x[:2]), ("block_tables", lambda x: x[:, :-1]),
    ("block_tables", lambda x: x.cpu()), ("block_tables", lambda x: x.t().contiguous().t()),
    ("sinks", lambda _: torch.zeros(7, device="cuda")), ("sinks", lambda _: torch.zeros(8, device="cuda").half()),
    ("out", lambda _: torch.zeros((3, 8, 128), device="cuda")),
    ("out", lambda _: torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")),
    ("out", lambda _: torch.zeros((3, 8, 256), dtype=torch.bfloat16, device="cuda")[..., :128]),
    ("lse", lambda _: torch.zeros((3, 7), device="cuda")), ("lse", lambda _: torch.zeros((8, 3), device="cuda").t()),
    ("workspace", lambda _: torch.zeros(1 << 22, dtype=torch.uint8)),
    ("workspace", lambda _: torch.zeros((1 << 11, 1 << 12), dtype=torch.uint8, device="cuda")[:, :1 << 11]),
])
def test_prefix_run_refuses(name, change):
    p, args, _ = prefix_case()
    args[name] = change(args.get(name))
    with pytest.raises(ValueError):
        api.paged_prefix_decode_run(p, **args)


def test_prefix_run_refuses_live_lengths_that_are_missing():
    c = make(**CASE)
    p = plan_of(c, freeze_seq_lens=False)
    run = lambda lens: api.paged_prefix_decode_run(p, c["q"], c["k"], c["v"], table(c), seq_lens_kv=lens)   # noqa: E731
    for lens in (torch.tensor(c["kv"][:2], dtype=torch.int32, device="cuda"), torch.tensor(c["kv"], device="cuda"),
                 torch.tensor(c["kv"] * 2, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            run(lens)
    with pytest.raises(L.PkaError) as e:
        run(None)
    assert e.value.code == L.PKA_ERR_INVALID_ARG


def test_workspaces():
    """One of the plan's size is enough, a smaller or unaligned one refused; two captured graphs
    and calls between them share one."""
    p, args, c = prefix_case()
    d = make([(7, [300, 20]), (3, [1, 2, 3])], heads=16, kv_heads=4, ps=32, seed=5)
    r = plan_of(d)
    n = max(p.workspace_bytes, r.workspace_bytes)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    run = lambda w: api.paged_prefix_decode_run(p, **args, workspace=w)   # noqa: E731
    for small in (ws[:p.workspace_bytes - 1], ws[:0]):
        with pytest.raises(L.PkaError) as e:
            run(small)
        assert e.value.code == L.PKA_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(L.PkaError) as e:
        run(ws[128:])
    assert e.value.code == L.PKA_ERR_INVALID_ARG
    first = run(ws[:p.workspace_bytes])
    other = lambda: api.paged_prefix_decode_run(r, d["q"], d["k"], d["v"], t, workspace=ws)   # noqa: E731
    t = table(d)
    second = other()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        a = run(ws)
    with torch.cuda.graph(graphs[1]):
        b = other()
    for i in (0, 1, 1, 0, 0, 1):
        for x in (*a, *b):
            x.fill_(7)
        graphs[i].replay()
        graphs[1 - i].replay()
        assert all(torch.equal(x, y) for x, y in zip((*a, *b), (*first, *second)))
        assert all(torch.equal(x, y) for x, y in zip(run(ws), first))
    want = ref.decode(d["q"], d["k"], d["v"], d["tables"], d["kv"], d["qo"], causal=False, scale=d["scale"])
    close(second, want, d["v"], d["dtype"], d["dtype"])
    p.check()
    r.check()


def rope_args():
    qkv = torch.randn((5, 8, 128), device="cuda").bfloat16()
    return dict(k=qkv[:, 4:6], v=qkv[:, 6:], slot_map=torch.arange(5, device="cuda"), q=qkv[:, :4],
                k_pages=torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16, device="cuda"),
                v_pages=torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16, device="cuda"),
                positions=torch.arange(5, dtype=torch.int32, device="cuda"),
                inv_freq=torch.ones(64, dtype=torch.float64, device="cuda"))


@pytest.mark.parametrize("name,change", [
    ("k", lambda x: x.half()), ("k", lambda x: x[:, :1]), ("k", lambda x: x[:4]), ("v", lambda x: x.contiguous()),
    ("q", lambda x: x[:4]), ("q", lambda x: x.float()), ("q", lambda x: x.cpu()), ("q", lambda x: x[..., :64]),
    ("q_out", lambda _: torch.zeros((5, 3, 128), dtype=torch.bfloat16, device="cuda")),
    ("slot_map", lambda x: x.int()), ("slot_map", lambda x: x[:4]), ("slot_map", lambda x: x.cpu()),
    ("slot_map", lambda x: x.repeat(2)[::2]), ("positions", lambda x: x.long()), ("positions", lambda x: x[:4]),
    ("positions", lambda x: x.expand(5, 5)), ("positions", lambda _: None), ("inv_freq", lambda x: x.float()),
    ("inv_freq", lambda x: x.repeat(2)[::2]), ("inv_freq", lambda _: None), ("k_pages", lambda x: x[:, :1]),
    ("v_pages", lambda x: x.half()), ("k_pages", lambda x: x.transpose(2, 3).contiguous().transpose(2, 3)),
    ("sections", lambda _: [32, 32]), ("pairs", lambda _: "both"),
    ("status", lambda _: torch.zeros(2, dtype=torch.int32, device="cuda")),
])
def test_rope_append_refuses(name, change):
    args = rope_args()
    pools = args["k_pages"], args["v_pages"]
    args[name] = change(args.get(name))
    with pytest.raises(ValueError):
        api.paged_rope_append(**args)
    torch.cuda.synchronize()
    assert not any(bool(x.any()) for x in pools)


@pytest.mark.parametrize("name,change", [
    ("kv_lens", lambda x: x.long()), ("kv_lens", lambda x: x[:2]), ("kv_lens", lambda x: x.cpu()),
    ("free_pages", lambda x: x.repeat(2)[::2]), ("free_head", lambda x: x.repeat(2)),
    ("block_tables", lambda x: x.t().contiguous().t()), ("block_tables", lambda x: x[0]),
    ("seq_lens", lambda _: torch.zeros(2, dtype=torch.int32, device="cuda")),
    ("status", lambda _: torch.zeros(1, device="cuda")),
])
@pytest.mark.parametrize("call", ["fork", "free", "compact"])
def test_page_operations_refuse(call, name, change):
    i32 = dict(dtype=torch.int32, device="cuda")
    args = dict(kv_lens=torch.tensor([20, 0, 5], **i32), free_pages=torch.arange(9, 20, **i32), free_head=torch.zeros(1, **i32),
                block_tables=torch.arange(9, **i32).view(3, 3))
    if call == "compact" and name == "seq_lens":
        name = "num_moves"
    args[name] = change(args.get(name))
    with pytest.raises(ValueError):
        if call == "fork":
            api.paged_kv_fork(torch.tensor([0], **i32), torch.tensor([1], **i32), page_size=16, **args)
        elif call == "free":
            api.paged_kv_free(torch.tensor([0], **i32), page_size=16, num_pages=20, **args)
        else:
            api.paged_kv_compact(page_size=16, num_pages=20, **args)
