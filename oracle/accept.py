"""Acceptance of drafted tokens in plain Python: the definition of dsa_tree_accept."""
from __future__ import annotations


def parent(mask, t):
    """The last token before t in the bit set mask[t]; mask None: a chain."""
    if mask is None:
        return t - 1
    below = mask[t] & ((1 << t) - 1)
    return below.bit_length() - 1


def accept(tok_start, masks, drafted, sampled, eos=-1):
    """masks: an integer of bits per token (of its sequence), or None.  (n_new, rows, tokens, next)."""
    n_new, rows, nxt = [], [], []
    for s0, s1 in zip(tok_start, tok_start[1:]):
        T, path, t = s1 - s0, [], 0
        mask = None if masks is None else masks[s0:s1]
        while t is not None and t < T:
            path.append(s0 + t)
            s = sampled[s0 + t]
            ends = s < 0 or s == eos
            t = None if ends else next((c for c in range(t + 1, T) if parent(mask, c) == t and drafted[s0 + c] == s), None)
        n_new.append(len(path))
        rows += path
        nxt.append(sampled[path[-1]] if path else -1)
    return n_new, rows, [sampled[r] for r in rows], nxt
