"""Paged decode in 64 bits, one request and KV head at a time."""

import math

import torch


def decode(q, k_pages, v_pages, tables, kv_lens, indptr, *, causal, scale, bmm2_scale=1.0, sinks=None):
    """(out, lse) in 64 bits; tables, kv_lens and indptr are lists."""
    H, Hkv, ps, D = q.shape[1], k_pages.shape[1], k_pages.shape[2], q.shape[2]
    G = H // Hkv
    out = torch.zeros((q.shape[0], H, D), dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0], H), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(kv_lens):
        ids = torch.tensor(tables[b][: -(-n // ps)], device=q.device)
        L = indptr[b + 1] - indptr[b]
        for h in range(Hkv):
            k, v = (p[ids, h].reshape(-1, D)[:n].double() for p in (k_pages, v_pages))
            for i in range(L):
                m = n - L + i + 1 if causal else n
                at = slice(h * G, (h + 1) * G)
                x = q[indptr[b] + i, at].double() @ k[:m].T * scale
                lse[indptr[b] + i, at] = torch.logsumexp(x, 1) / math.log(2.0)
                total = torch.logsumexp(x, 1)
                if sinks is not None:
                    total = torch.logaddexp(total, sinks[at].double())
                out[indptr[b] + i, at] = torch.exp(x - total[:, None]) @ v[:m] * bmm2_scale
    return out, lse
