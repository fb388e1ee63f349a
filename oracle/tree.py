"""Attention of drafted tokens over a paged cache in fp64 (torch): the definition.

One token at a time over the list of keys that it sees; nothing that it does not
see is read.
"""
from __future__ import annotations

import torch


def seen_by(mask, t0, t, T):
    """Drafted tokens that token t (of its sequence) sees: bits of mask[t0 + t], or 0..t."""
    if mask is None:
        return list(range(t + 1))
    words = [int(w) & ((1 << 64) - 1) for w in mask[t0 + t].tolist()]
    return [j for j in range(T) if (words[j // 64] >> (j % 64)) & 1]


def tree_attn(q, pool, table, lens, kv_new, tok_start, mask, scale, d_v):
    """(out, m, l, A, S) for every token with a sequence: A[t, h] = sum p |v| / l per value
    column and S[t, h] = max_s scale * sum_d |q_d k_d| carry the error bounds.  Tokens without
    one keep NaN.  table / lens / tok_start: lists; a page outside the pool counts as unseen."""
    n, H, d = q.shape
    R = pool.shape[1]
    dev = q.device
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.float64, device=dev)
    out, A = nan(n, H, d_v), nan(n, H, d_v)
    m, l, S = nan(n, H), nan(n, H), nan(n, H)
    for b, length in enumerate(lens):
        t0, t1 = tok_start[b], tok_start[b + 1]
        if t0 == t1:
            continue
        pos = [s for s in range(length) if 0 <= table[b][s // R] < pool.shape[0]]
        pages = torch.tensor([table[b][s // R] for s in pos], dtype=torch.long, device=dev)
        cached = pool[pages, torch.tensor([s % R for s in pos], dtype=torch.long, device=dev)].double()
        for t in range(t1 - t0):
            js = [t0 + j for j in seen_by(mask, t0, t, t1 - t0)]
            k = torch.cat([cached, kv_new[js].double()]) if js else cached
            r = t0 + t
            if k.shape[0] == 0:
                out[r], A[r], m[r], l[r], S[r] = 0, 0, -float("inf"), 0, 0
                continue
            qt = q[r].double()
            x = scale * (qt @ k.T)                                   # [H, keys]
            m[r] = x.max(-1).values
            p = torch.exp(x - m[r][:, None])
            l[r] = p.sum(-1)
            out[r] = (p @ k[:, :d_v]) / l[r][:, None]
            A[r] = (p @ k[:, :d_v].abs()) / l[r][:, None]
            S[r] = scale * (qt.abs() @ k.abs().T).max(-1).values
    return out, m, l, A, S
