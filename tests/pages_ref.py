"""Page operations and rotations in plain Python and 64 bits, the tests' reference."""

import torch


def fork(parents, children, kv, free, head, tables, ps):
    """(tables, seq_lens, src, dst, head) of lists; tables is copied."""
    tables, seq = [list(r) for r in tables], list(kv)
    src, dst = [], []
    for p, c in zip(parents, children):
        full = kv[p] // ps
        tables[c][:full] = tables[p][:full]
        s = d = -1
        if kv[p] % ps:
            s, d = tables[p][full], free[head]
            tables[c][full] = d
            head += 1
        src.append(s)
        dst.append(d)
        seq[c] = kv[p]
    return tables, seq, src, dst, head


def held(kv, tables, ps, rows):
    out = set()
    for b in rows:
        out |= set(tables[b][: -(-kv[b] // ps)])
    return out


def release(rows, kv, free, head, tables, ps):
    """(free, seq_lens, head)."""
    gone = held(kv, tables, ps, rows) - held(kv, tables, ps, set(range(len(kv))) - set(rows))
    free = list(free)
    free[head - len(gone):head] = sorted(gone)
    return free, [0 if b in set(rows) else n for b, n in enumerate(kv)], head - len(gone)


def compact(kv, free, head, tables, ps):
    """(tables, free, src, dst)."""
    used, opened = held(kv, tables, ps, range(len(kv))), set(free[head:])
    every = sorted(used | opened)
    low = set(every[: len(used)])
    src, dst = sorted(used - low), sorted(opened & low)
    to = dict(zip(src, dst))
    new = [[to.get(p, p) if j < -(-kv[b] // ps) else p for j, p in enumerate(r)]
           for b, r in enumerate(tables)]
    return new, list(free[:head]) + every[len(used):], src, dst


def rotate(x, positions, inv_freq, sections, pairs):
    """Rows ``x`` [T, H, D] rotated in 64 bits; positions [axes, T]."""
    y = x.double().clone()
    half = inv_freq.numel()
    j = 0
    for axis, count in enumerate(sections):
        for _ in range(count):
            i0, i1 = (j, j + half) if pairs == "halves" else (2 * j, 2 * j + 1)
            angle = positions[axis].double() * inv_freq[j].double()
            c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            a, b = x[..., i0].double(), x[..., i1].double()
            y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
            j += 1
    assert j == half
    return y
