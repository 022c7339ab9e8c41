"""What the rotated append takes and refuses on the host, beyond single arguments (no GPU needed).

A call that is taken would go on to the launch; without a GPU that fails with PKA_ERR_CUDA, and where
there is one nothing may run at these addresses, so such calls are made without a GPU only."""

import random

import pytest
import torch

from paged_kv_attention_32_gb300 import _lib as L
from tests.test_pages_binding import rope


def test_no_tokens_need_no_positions():
    """The address of an empty tensor is NULL."""
    none = dict(T=0, k=None, v=None, slots=None, pos=None, kp=None, vp=None)
    assert rope(**none) == L.PKA_OK
    assert rope(**none, Hq=0, q=None, q_out=None) == L.PKA_OK
    # what the call would rotate by is looked at all the same
    for kw in (dict(freq=None), dict(sections=None), dict(axes=0), dict(pairs=2)):
        assert rope(**(none | kw)) == L.PKA_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run at these addresses")
def test_one_row_of_positions_for_all_axes():
    assert rope(pos_row=0) == rope(pos_row=8) == L.PKA_ERR_CUDA
    assert rope(pos_row=1) == rope(pos_row=-8) == L.PKA_ERR_INVALID_ARG


def rows_meet(n, outer, m, inner, row):
    """By listing all rows."""
    starts = sorted(i * outer + j * inner for i in range(n) for j in range(m))
    return any(b - a < row for a, b in zip(starts, starts[1:]))


# tokens, token stride, heads, head stride of q_out (rows of 128), or pages and heads of pools (rows of 2048)
LAYOUTS = [
    (5, 128, 3, 128), (5, 256, 3, 128), (5, 384, 3, 128), (5, 392, 3, 128), (3, 128, 5, 384), (3, 128, 5, 256),
    (4, 256, 4, 384), (3, 256, 3, 384), (2, 256, 5, 384), (4, 640, 3, 256), (4, 120, 1, 0), (1, 0, 4, 120),
    (1, 0, 4, 128), (4, 128, 1, 0), (1, 8, 1, 8), (2, 0, 3, 128), (3, 128, 2, 0), (3, 136, 2, 4096), (100, 130 * 8, 9, 128),
]


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run at these addresses")
@pytest.mark.parametrize("pools", [False, True])
def test_rows_written_twice(pools):
    """Outputs are refused where two of their rows share an element, and nowhere else."""
    r = random.Random(3)
    drawn = [(r.randint(1, 7), 8 * r.randint(0, 160), r.randint(1, 7), 8 * r.randint(0, 160)) for _ in range(400)]
    seen = set()
    for n, outer, m, inner in LAYOUTS + drawn:
        if pools:
            outer, inner = 16 * outer, 16 * inner
            kw = dict(Hq=0, q=None, q_out=None, Hkv=m, pages=n, page=outer, head=inner, kp=1 << 40, vp=1 << 50)
            want = rows_meet(n, outer, m, inner, 2048)
        else:
            kw = dict(T=n, Hq=m, q_out=1 << 40, o_tok=outer, o_head=inner)
            want = rows_meet(n, outer, m, inner, 128)
        code = rope(**kw)
        assert (code == L.PKA_ERR_INVALID_ARG) == want, (n, outer, m, inner, code)
        seen.add(want)
    assert seen == {True, False}


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run at these addresses")
def test_rows_of_the_largest_layouts():
    """Strides and counts whose products pass 64 bits, and the longest search."""
    far = dict(Hq=0, q=None, q_out=None, kp=1 << 40, vp=1 << 50)
    assert rope(**far, pages=2 ** 31 - 1, Hkv=65536, page=2 ** 62, head=2 ** 61) == L.PKA_ERR_INVALID_ARG
    assert rope(**far, pages=2 ** 31 - 1, Hkv=3, page=2 ** 62, head=2 ** 60) != L.PKA_ERR_INVALID_ARG
    # heads a page and a half apart over pages: rows meet only where three pages are two heads
    assert rope(**far, pages=2 ** 31 - 1, Hkv=65536, page=4096, head=6144) == L.PKA_ERR_INVALID_ARG
    assert rope(**far, pages=3, Hkv=65536, page=4096, head=6144) != L.PKA_ERR_INVALID_ARG


def starts(at, n, outer, m, inner):
    return [at + i * outer + j * inner for i in range(n) for j in range(m)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run at these addresses")
def test_pools_that_share_rows():
    """Key and value pools are refused where a page's rows of the one are rows of the other, and taken where
    they lie between each other: halves of a page, of a head, of the whole, alternating heads."""
    r = random.Random(5)
    row = 2048   # 16 slots of 128 values
    seen = set()
    named = [(5, 2 * 3 * row, 3, row, 3 * row, False), (5, 6 * row, 3, 2 * row, row, False), (5, 3 * row, 3, row, 15 * row, False),
             (4, row, 3, 8 * row, 4 * row, False), (4, 2 * row, 3, 8 * row, row, False),
             (5, 3 * row, 3, row, 12 * row, True), (5, 3 * row, 3, row, row, True), (5, 3 * row, 3, row, 8, True),
             (5, 6 * row, 3, row, 3 * row - 8, True), (1, 0, 1, 0, row, False), (1, 8, 1, 8, row - 8, True)]
    named += [
        (r.randint(1, 6), r.choice([128, 8, 1]) * 8 * r.randint(0, 200), r.randint(1, 6),
         r.choice([128, 8, 1]) * 8 * r.randint(0, 200), r.choice([128, 8, 1]) * 8 * r.randint(-400, 400), None)
        for _ in range(3000)]
    for n, outer, m, inner, at, meet in named:
        if rows_meet(n, outer, m, inner, row):
            continue
        k, v = sorted(starts(0, n, outer, m, inner)), starts(at, n, outer, m, inner)
        want = any(abs(x - y) < row for x in k for y in v)
        assert meet is None or meet == want
        base = 1 << 40
        code = rope(Hq=0, q=None, q_out=None, Hkv=m, pages=n, page=outer, head=inner, kp=base, vp=base + 2 * at)
        assert (code == L.PKA_ERR_INVALID_ARG) == want, (n, outer, m, inner, at, code)
        seen.add(want)
    assert seen == {True, False}


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is taken would run at these addresses")
def test_inputs_among_what_is_written():
    """Inputs in a pool or under q_out are refused, by the byte; those in the gaps between rows are taken,
    and so is q_out over all of q."""
    def spans(at, n, outer, m, inner, size):
        return [(x, x + size) for x in starts(at, n, 2 * outer, m, 2 * inner)]

    r = random.Random(7)
    K, V, Q, base = 1 << 40, 1 << 41, 1 << 42, 1 << 43   # apart from each other and from all else
    seen = {}
    for turn in range(6000):
        T, Hq, Hkv, pages = (r.randint(1, 4) for _ in range(4))
        step = lambda row: 8 * r.choice([row // 8, r.randint(row // 8, row // 2)])   # noqa: E731
        page, head = (16 * 128 * Hkv + 8 * r.randint(0, 400), 16 * 128) if r.random() < 0.5 else (
            16 * 128, 16 * 128 * pages + 8 * r.randint(0, 400))
        kw = dict(T=T, Hq=Hq, Hkv=Hkv, pages=pages, page=page, head=head, kp=K, vp=V, q=base, k=base + (1 << 24),
                  v=base + (2 << 24), pos=base + (3 << 24), freq=base + (4 << 24), slots=base + (5 << 24),
                  status=base + (6 << 24), q_out=Q, axes=2, pos_row=T + r.randint(0, 9))
        kw["q_head"], kw["o_head"], kw["kv_head"] = step(128), step(128), step(128)
        for tok, h, n in (("q_tok", "q_head", Hq), ("o_tok", "o_head", Hq), ("kv_tok", "kv_head", Hkv)):
            kw[tok] = kw[h] * (n - 1) + step(128)
        name, align = r.choice([("q", 16), ("k", 16), ("v", 16), ("pos", 4), ("freq", 8), ("slots", 8), ("status", 4),
                                ("q_out", 16)])
        into = r.choice([K, V, Q])
        if name == "q_out" and into == Q:
            into = kw[r.choice("qkv")]
        span = 2 * (kw["o_tok"] * T if into == Q else page * pages + head * Hkv if into in (K, V) else 512 * T)
        kw[name] = into + align * r.randint(-40, span // align)
        if turn % 20 == 0:   # in place, with k and v beside q in a fused projection, or a row too far in
            kw.update(q=base, q_out=base, k=base + 256 * Hq - 256 * (turn % 40 == 0), v=base + 256 * (Hq + Hkv), o_head=128,
                      q_head=128, kv_head=128, pos=base + (3 << 24), freq=base + (4 << 24), slots=base + (5 << 24),
                      status=base + (6 << 24), **{x: 128 * (Hq + 2 * Hkv) for x in ("q_tok", "o_tok", "kv_tok")})
            name = "fused"
        ins = {"q": spans(kw["q"], T, kw["q_tok"], Hq, kw["q_head"], 256),
               "k": spans(kw["k"], T, kw["kv_tok"], Hkv, kw["kv_head"], 256),
               "v": spans(kw["v"], T, kw["kv_tok"], Hkv, kw["kv_head"], 256),
               "pos": [(kw["pos"] + 4 * a * kw["pos_row"], kw["pos"] + 4 * a * kw["pos_row"] + 4 * T) for a in (0, 1)],
               "freq": [(kw["freq"], kw["freq"] + 512)], "slots": [(kw["slots"], kw["slots"] + 8 * T)],
               "status": [(kw["status"], kw["status"] + 4)]}
        pools = [spans(x, pages, page, Hkv, head, 4096) for x in (K, V)]
        out = spans(kw["q_out"], T, kw["o_tok"], Hq, kw["o_head"], 256)
        if (kw["q"], kw["q_tok"], kw["q_head"]) == (kw["q_out"], kw["o_tok"], kw["o_head"]):
            pairs = [(x, out) for n, x in ins.items() if n != "q"]
        else:
            pairs = [(x, out) for x in ins.values()]
        pairs += [(x, p) for x in (out, *ins.values()) for p in pools]
        want = any(a < d and c < b for x, y in pairs for a, b in x for c, d in y)
        code = rope(**kw)
        assert (code == L.PKA_ERR_INVALID_ARG) == want, (kw, code)
        seen.setdefault(name, set()).add(want)
    assert all(x == {True, False} for x in seen.values()) and len(seen) == 9
