"""Acceptance of drafted tokens on the GPU against the definition (whole numbers: equal)."""
import random

import pytest
import torch

from gpu_util import DEV, lib
from oracle.accept import accept

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def words_of(masks, words):
    rows = [[(m >> (64 * w)) & ((1 << 64) - 1) for w in range(words)] for m in masks]
    return torch.tensor([[v - (1 << 64) if v >> 63 else v for v in r] for r in rows], dtype=torch.int64, device=DEV)


def trees(rng, counts, tree, match, vocab=50):
    """Random trees (or chains) with tokens that often match; some twins, some further roots."""
    masks, drafted, sampled, at = [], [], [], 0
    for T in counts:
        rows = []
        sampled += [rng.randrange(vocab) for _ in range(T)]
        for t in range(T):
            p = -1 if t == 0 or (tree and rng.random() < 0.05) else rng.randrange(max(0, t - 6), t) if tree else t - 1
            rows.append((1 << t) | (rows[p] if p >= 0 else 0))
            drafted.append(sampled[at + p] if p >= 0 and rng.random() < match else rng.randrange(vocab))
        masks += rows
        at += T
    return masks, drafted, sampled


def run(dsa, starts, masks, drafted, sampled, eos=-1, words=0, room=0, stream=None):
    n, total = len(starts) - 1, len(drafted) + room
    pad = [0] * room
    c = dsa.make_cache(n_seqs=n, n_pages=1, page_rows=1, max_pages=1)
    t = dsa.make_tree(n_tok=total, H=1, d_qk=1, d_v=1, scale=1.0, mask_words=words)
    o = [torch.full((k,), 77, dtype=torch.int32, device=DEV) for k in (n, total, total, n)]
    dsa.tree_accept(c, t, ints(starts), words_of(masks + pad, words) if words else None, ints(drafted + pad),
                    ints(sampled + pad), *o, eos=eos, stream=stream)
    torch.cuda.synchronize()
    return [x.tolist() for x in o]


def check(dsa, counts, tree, match=0.7, seed=0, eos=-1, room=0):
    masks, drafted, sampled = trees(random.Random(seed), counts, tree, match)
    starts = [0]
    for T in counts:
        starts.append(starts[-1] + T)
    words = -(-max(counts) // 64) if tree else 0
    got = run(dsa, starts, masks, drafted, sampled, eos, words, room)
    n_new, rows, tokens, nxt = accept(starts, masks if tree else None, drafted, sampled, eos)
    behind = [-1] * (len(drafted) + room - len(rows))
    assert got == [n_new, rows + behind, tokens + behind, nxt]
    assert dsa.get_status() == 0


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("counts", [[1], [2], [5], [64], [65], [130], [0, 3, 0, 1, 0], [300, 1, 200], [31] * 31, [7] * 32,
                                    [3] * 33, list(range(70))])
def test_trees_and_chains(counts, tree):
    dsa = lib()
    for seed, match in ((1, 0.0), (2, 0.7), (3, 0.95), (4, 1.0)):
        check(dsa, counts, tree, match, seed, eos=random.Random(seed).choice([-1, 7]), room=seed % 3)


@pytest.mark.parametrize("n", [256, 257, 300, 1000, 8192])
def test_many_sequences(n):
    dsa = lib()
    rng = random.Random(n)
    check(dsa, [rng.randrange(0, 9) for _ in range(n)], True, 0.9, n)
    check(dsa, [rng.randrange(0, 3) for _ in range(n)], False, 0.9, n, room=5)


def test_negative_tokens_end_a_sequence():
    dsa = lib()
    got = run(dsa, [0, 3], [], [5, -1, -1], [-1, -1, 4])
    assert got == [[1], [0, -1, -1], [-1, -1, -1], [-1]]


def test_numbers_out_of_range():
    dsa = lib()
    E = dsa.DSA_ERR_INDEX
    # sequence 1 ends before it begins; sequence 2 goes past the last token
    got = run(dsa, [0, 2, 1, 9], [], [1, 2, 3, 4], [2, 5, 4, 6])
    assert dsa.get_status() == E and got[0] == [2, 0, 0] and got[3] == [5, -1, -1]
    assert got[1] == [0, 1, -1, -1] and got[2] == [2, 5, -1, -1]
    assert run(dsa, [-1, 2], [], [1, 2], [2, 3])[0] == [0] and dsa.get_status() == E
    # more tokens than the mask has bits for
    got = run(dsa, [0, 65], [1] * 65, [1] * 65, [1] * 65, words=1)
    assert dsa.get_status() == E and got[0] == [0]
    # bounds that overlap name the same tokens more than once: nothing is written past the end
    got = run(dsa, [0, 2, 0, 2, 0, 2], [], [1, 2], [2, 3])
    assert dsa.get_status() == E and got[1] == [0, 1] and got[0] == [2, 0, 2, 0, 2]


def test_masks_that_see_later_or_missing_tokens():
    # bits at and above a token, and of tokens that its sequence does not have, mean nothing
    dsa = lib()
    rng = random.Random(5)
    masks, drafted, sampled = trees(rng, [20] * 6, True, 0.9)
    starts = [20 * i for i in range(7)]
    noisy = [m | (rng.getrandbits(64) << (i % 20)) & ((1 << 64) - 1) for i, m in enumerate(masks)]
    want = accept(starts, masks, drafted, sampled)
    got = run(dsa, starts, noisy, drafted, sampled, words=1)
    assert got[0] == want[0] and got[3] == want[3] and got[1][:len(want[1])] == want[1]


def test_graph_replay_and_other_stream():
    dsa = lib()
    counts = [9] * 40
    starts = [9 * i for i in range(41)]
    c = dsa.make_cache(n_seqs=40, n_pages=1, page_rows=1, max_pages=1)
    t = dsa.make_tree(n_tok=360, H=1, d_qk=1, d_v=1, scale=1.0, mask_words=1)
    m = torch.zeros(360, 1, dtype=torch.int64, device=DEV)
    d, s, st = ints([0] * 360), ints([0] * 360), ints(starts)
    o = [ints([0] * k) for k in (40, 360, 360, 40)]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        dsa.tree_accept(c, t, st, m, d, s, *o)
    for seed in range(3):
        masks, drafted, sampled = trees(random.Random(seed), counts, True, 0.8)
        m.copy_(words_of(masks, 1))
        d.copy_(ints(drafted))
        s.copy_(ints(sampled))
        g.replay()
        torch.cuda.synchronize()
        want = accept(starts, masks, drafted, sampled)
        assert o[0].tolist() == want[0] and o[3].tolist() == want[3]
        assert o[1].tolist() == want[1] + [-1] * (360 - len(want[1]))
    assert run(dsa, starts, masks, drafted, sampled, words=1, stream=side)[0] == want[0]


def test_refused_tensors():
    dsa = lib()
    c = dsa.make_cache(n_seqs=2, n_pages=1, page_rows=1, max_pages=1)
    t = dsa.make_tree(n_tok=4, H=1, d_qk=1, d_v=1, scale=1.0)
    st, v = ints([0, 2, 4]), lambda n: ints([0] * n)
    ok = dict(tok_start=st, mask=None, drafted=v(4), sampled=v(4), n_new=v(2), row_index=v(4), tokens=v(4), next_token=v(2))
    dsa.tree_accept(c, t, **ok)
    for e, kw in ((ValueError, dict(tok_start=v(2))), (TypeError, dict(drafted=v(4).long())), (ValueError, dict(sampled=v(5))),
                  (ValueError, dict(n_new=v(4)[::2])), (ValueError, dict(row_index=v(3))), (ValueError, dict(tokens=v(4).cpu())),
                  (TypeError, dict(next_token=None))):
        with pytest.raises(e):
            dsa.tree_accept(c, t, **dict(ok, **kw))
    masked = dsa.make_tree(n_tok=4, H=1, d_qk=1, d_v=1, scale=1.0, mask_words=1)
    for kw in (dict(t=masked), dict(row_index=ok["tokens"]), dict(n_new=ok["next_token"]), dict(tokens=ok["drafted"]), dict(eos=-2)):
        with pytest.raises(dsa.DSAError) as e:
            dsa.tree_accept(c, **{**dict(t=t), **ok, **kw})
        assert e.value.code == dsa.DSA_ERR_INVALID_ARG
    assert dsa.get_status() == 0
