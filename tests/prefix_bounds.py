"""Attention behind shared prefixes in 64 bits together with how far the kernels may be from it.

With p the weights of a row, summing to 1, and A = sum p |v| for each output element:

  * p is rounded to the input type before the product with v: half a step of each, so u A at most,
    u = finfo(type).eps / 2.  In f16 a weight below the smallest normal number is off by 2^-25 of the largest
    instead: 2^-25 sum |v| / sum exp(s - max);
  * scores: eight 32-bit additions of 16 products (each at most a step, 2^-23, of sum |q k|), one rounding each of
    the scaled score and of what goes to exp2, which is off by 2^-22: for scores whose products stay below 16
    that is 2^-16 of p, and again of the sum that it is divided by;
  * sums over the N keys of a piece, which has accumulators of its own: N / 16 additions in each, off by at most a
    step of A, and N / 64 + 64 of the row's sum, half a step each;
  * joining the states and the last scaling: fewer than 64 roundings of 2^-24;
  * one rounding to the output type.
"""

import math

import torch


def decode(q, k_pages, v_pages, tables, kv_lens, indptr, *, causal, scale, dtype, out_dtype, piece):
    """(out, lse, allowed error of out), in 64 bits; tables, kv_lens and indptr are lists, `piece` the keys of the
    longest piece."""
    H, Hkv, ps, D = q.shape[1], k_pages.shape[1], k_pages.shape[2], q.shape[2]
    G = H // Hkv
    out, allowed = (torch.zeros((q.shape[0], H, D), dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full((q.shape[0], H), -math.inf, dtype=torch.float64, device=q.device)
    u, u_out = (torch.finfo(t).eps / 2 for t in (dtype, out_dtype))
    for b, n in enumerate(kv_lens):
        ids = torch.tensor(tables[b][: -(-n // ps)], device=q.device)
        L = indptr[b + 1] - indptr[b]
        for h in range(Hkv):
            k, v = (p[ids, h].reshape(-1, D)[:n].double() for p in (k_pages, v_pages))
            at = slice(h * G, (h + 1) * G)
            for i in range(L):
                m, row = (n - L + i + 1 if causal else n), indptr[b] + i
                x = q[row, at].double() @ k[:m].T * scale
                assert float((q[row, at].double().abs() @ k[:m].T.abs()).max()) * abs(scale) < 16
                lse[row, at] = torch.logsumexp(x, 1) / math.log(2.0)
                p = torch.softmax(x, 1)
                out[row, at] = p @ v[:m]
                mean = p @ v[:m].abs()
                rel = u + 2 * 2.0 ** -16 + piece / 16 * 2.0 ** -23 + (piece / 64 + 128) * 2.0 ** -24
                allowed[row, at] = rel * mean + u_out * out[row, at].abs()
                if dtype == torch.float16:
                    allowed[row, at] += 2.0 ** -25 * p.amax(1, keepdim=True) * v[:m].abs().sum(0)
    return out, lse, allowed
