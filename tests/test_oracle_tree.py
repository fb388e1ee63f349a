"""The fp64 definition of the drafted-tree attention against plain dense attention and by hand."""
import math

import torch

from oracle.tree import seen_by, tree_attn


def test_masks_name_drafted_tokens_across_words():
    mask = torch.zeros(3, 2, dtype=torch.int64)
    mask[2, 0] = -(1 << 63)   # bit 63
    mask[2, 1] = 1            # bit 64
    assert seen_by(mask, 1, 1, 65) == [63, 64]
    assert seen_by(mask, 1, 1, 64) == [63] and seen_by(mask, 0, 0, 5) == []
    assert seen_by(None, 7, 2, 5) == [0, 1, 2]


def test_hand_worked():
    # one cached row k = (0, 1), one drafted row d = (ln 3, 2), q = (1, 0), scale 1, d_v = 2:
    # logits 0 and ln 3, so p = 1/4, 3/4
    q = torch.tensor([[[1.0, 0.0]]])
    pool, new = torch.tensor([[[0.0, 1.0]]]), torch.tensor([[math.log(3.0), 2.0]])
    out, m, l, A, S = tree_attn(q, pool, [[0]], [1], new, [0, 1], None, 1.0, 2)
    assert torch.allclose(out[0, 0], torch.tensor([0.75 * math.log(3.0), 1.75], dtype=torch.float64), atol=1e-6)
    assert abs(float(m) - math.log(3.0)) < 1e-6 and abs(float(l) - 4 / 3) < 1e-6


def test_chain_is_causal_attention_and_empty_rows_are_zero():
    g = torch.Generator().manual_seed(1)
    T, H, d, n = 5, 3, 8, 6
    q, new = torch.randn(T, H, d, generator=g), torch.randn(T, d, generator=g)
    pool = torch.randn(4, 3, d, generator=g)
    table = [[2, 0]]
    out, m, l, _, _ = tree_attn(q, pool, table, [n], new, [0, T], None, 0.3, d)
    k = torch.cat([pool[2], pool[0], new]).double()
    x = 0.3 * torch.einsum("thd,sd->ths", q.double(), k)
    hidden = torch.arange(n + T)[None, :] > n + torch.arange(T)[:, None]
    x = x.masked_fill(hidden[:, None, :], -math.inf)
    assert torch.allclose(out, torch.softmax(x, -1) @ k)
    assert torch.allclose(m + l.log(), torch.logsumexp(x, -1))
    out, m, l, _, _ = tree_attn(q, pool, [[9, 9]], [n], new, [0, T], torch.zeros(T, 1, dtype=torch.int64), 0.3, d)
    assert not out.any() and not l.any() and (m == -math.inf).all()
