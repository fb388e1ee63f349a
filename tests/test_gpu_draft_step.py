"""A step of generation with drafted trees, as a server makes it: rotary positions, attention over the
paged cache, sampling at every drafted position, acceptance, new rows of the cache; eagerly and as a
replayed graph.

The model is a table: a token's query and kv row are table entries (rotated at its position), the
logits a product of the attention's result.  Sampled tokens must be those of the definition on the logits
that the step computed, accepted ones those of the definition; the cache must hold, bit for bit, the
rotated rows of each sequence's own tokens at their own positions.
"""
import random

import pytest
import torch

from gpu_util import DEV, lib
from oracle.accept import accept
from oracle.rope import frequencies, rope
from oracle.sample import sample
from oracle.tree import tree_attn

pytestmark = pytest.mark.gpu
H, D, DV, ROT, V, SCALE = 16, 576, 512, 64, 997, 192 ** -0.5
N, T, P, R, M = 5, 6, 64, 16, 10                 # sequences, drafted tokens of each, pages, rows of a page, pages of a sequence
PARENT = [-1, 0, 0, 1, 1, 3]                     # the tree of drafts
DEPTH = [0, 1, 1, 2, 2, 3]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    def __init__(self, dsa):
        g = torch.Generator().manual_seed(7)
        bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)
        self.dsa = dsa
        self.e_q, self.e_kv, self.w_out = bf(V, H, D) * 0.5, bf(V, D), bf(H * DV, V) * 0.05
        self.rope = dsa.make_rope(rot_dim=ROT, parts=[dsa.rope_part(heads=H, dim=D, offset=DV),
                                                      dsa.rope_part(heads=1, dim=D, offset=DV)])
        n_tok = N * T
        self.cache = dsa.make_cache(n_seqs=N, n_pages=P, page_rows=R, max_pages=M)
        self.tree = dsa.make_tree(n_tok=n_tok, H=H, d_qk=D, d_v=DV, scale=SCALE, mask_words=1)
        self.sampler = dsa.make_sampler(rows=n_tok, vocab=V, requests=N)
        self.pool = torch.zeros(P, R, D, dtype=torch.bfloat16, device=DEV)
        self.table, self.lens, self.refs = ints([[0] * M] * N), ints([0] * N), ints([0] * P)
        self.start = ints([T * b for b in range(N + 1)])
        bits = [0] * T
        for t in range(T):
            bits[t] = (1 << t) | (bits[PARENT[t]] if t else 0)
        self.bits = bits
        self.mask = torch.tensor(bits * N, dtype=torch.int64, device=DEV).view(n_tok, 1)
        self.request = ints([b for b in range(N) for _ in range(T)])
        self.depth = ints(DEPTH * N)
        self.temperature = torch.tensor([0.0, 0.5, 1.0, 0.8, 0.7], device=DEV)
        self.top_k, self.top_p = ints([0, 3, 0, 40, 0]), torch.tensor([1.0, 1.0, 0.6, 0.9, 0.95], device=DEV)
        self.drafted, self.u = ints([0] * n_tok), torch.zeros(n_tok, device=DEV)
        self.sampled, self.prob = ints([0] * n_tok), torch.zeros(n_tok, device=DEV)
        self.n_new, self.rows, self.tokens, self.next = ints([0] * N), ints([0] * n_tok), ints([0] * n_tok), ints([0] * N)
        self.slots = ints([0] * n_tok)
        self.out = torch.zeros(n_tok, H, DV, dtype=torch.bfloat16, device=DEV)
        self.m, self.l = torch.zeros(n_tok, H, device=DEV), torch.zeros(n_tok, H, device=DEV)
        self.ws = torch.zeros(dsa.tree_workspace_size(self.cache, self.tree), dtype=torch.uint8, device=DEV)

    def forward(self):
        d, tok = self.dsa, self.drafted.long()
        self.pos = (self.lens[self.request.long()] + self.depth).int()
        self.q_raw, self.kv_raw = self.e_q[tok], self.e_kv[tok]
        self.q, self.kv = torch.empty_like(self.q_raw), torch.empty_like(self.kv_raw)
        d.rope_apply(self.rope, self.pos, (self.q_raw, self.kv_raw), (self.q, self.kv))
        d.tree_attn_fwd(self.cache, self.tree, self.q, self.pool, self.table, self.lens, self.kv, self.start, self.mask,
                        self.out, self.m, self.l, self.ws)
        self.logits = self.out.view(N * T, H * DV) @ self.w_out
        d.sample(self.sampler, self.logits, self.u, self.temperature, self.top_k, self.top_p, None, self.request,
                 self.sampled, self.prob)

    def keep(self):
        d = self.dsa
        d.tree_accept(self.cache, self.tree, self.start, self.mask, self.drafted, self.sampled, self.n_new, self.rows,
                      self.tokens, self.next)
        d.cache_extend(self.cache, self.n_new, self.table, self.lens, self.refs, self.lens, self.refs, self.slots)
        d.cache_write(self.cache, self.pool, self.kv, self.slots, self.rows)

    def draft(self, rng, last):
        """Drafts that are partly right: child 1 of each kept token is what the model will sample there (the
        logits of a token do not depend on its children)."""
        drafted = [x for b in range(N) for x in [last[b]] + [rng.randrange(V) for _ in range(T - 1)]]
        self.u.copy_(torch.tensor([rng.random() for _ in range(N * T)]))
        for level in range(3):
            self.drafted.copy_(ints(drafted))
            self.forward()
            s = self.sampled.tolist()
            for b in range(N):
                for t in range(T):
                    if DEPTH[t] == level + 1 and (b + t + level) % 3:
                        drafted[b * T + t] = s[b * T + PARENT[t]]
        self.drafted.copy_(ints(drafted))
        return drafted


def check_step(s, hist, lens):
    """The step's parts against their definitions; returns the kept rows."""
    dsa, tok = s.dsa, s.drafted.tolist()
    assert dsa.get_status() == 0
    pos = [lens[b] + DEPTH[t] for b in range(N) for t in range(T)]
    assert s.pos.tolist() == pos
    f = frequencies(ROT)
    for got, raw in ((s.q, s.q_raw), (s.kv.view(-1, 1, D), s.kv_raw.view(-1, 1, D))):
        want = rope(raw, pos, f, DV, "interleaved")
        # bf16 rounds by half a step; cosine and sine are good to 2^-21
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * raw.double().abs().max()).all())
    settings = list(zip(s.temperature.tolist(), s.top_k.tolist(), s.top_p.tolist()))
    x, u = s.logits.double().cpu().numpy(), s.u.tolist()
    for r in range(N * T):
        want, p, margin = sample(x[r], u[r], *settings[r // T])
        assert margin > 2.0 ** -27 and s.sampled[r] == want and abs(float(s.prob[r]) - p) <= p * 2.0 ** -23
    n_new, rows, tokens, nxt = accept(s.start.tolist(), s.bits * N, tok, s.sampled.tolist())
    behind = [-1] * (N * T - len(rows))
    assert [s.n_new.tolist(), s.rows.tolist(), s.tokens.tolist(), s.next.tolist()] == [n_new, rows + behind, tokens + behind, nxt]
    at = 0
    for b in range(N):
        hist[b] += [tok[r] for r in rows[at:at + n_new[b]]]
        at += n_new[b]
    assert s.lens.tolist() == [len(h) for h in hist]
    table = s.table.tolist()
    for b, h in enumerate(hist):
        # the sequence's own tokens, each rotated at its place
        rows_b = s.e_kv[torch.tensor(h, device=DEV)].clone()
        r1 = dsa.make_rope(rot_dim=ROT, parts=[dsa.rope_part(heads=1, dim=D, offset=DV)])
        dsa.rope_apply(r1, torch.arange(len(h), dtype=torch.int32, device=DEV), (rows_b,))
        i = torch.tensor([table[b][j // R] * R + j % R for j in range(len(h))], device=DEV)
        assert torch.equal(s.pool.view(-1, D)[i].view(torch.int16), rows_b.view(torch.int16))
    return n_new, nxt


def test_drafted_steps():
    dsa = lib()
    s, rng = Server(dsa), random.Random(5)
    hist, last, kept = [[] for _ in range(N)], [3, 14, 159, 26, 535], []
    for step in range(6):
        lens = s.lens.tolist()
        s.draft(rng, last)
        s.forward()
        if step == 3:
            ref = tree_attn(s.q, s.pool, s.table.tolist(), lens, s.kv, s.start.tolist(), s.mask,
                            float(torch.tensor(SCALE)), DV)[0]
            assert float((s.out.double() - ref).abs().max()) < 2e-2
        s.keep()
        torch.cuda.synchronize()
        n_new, last = check_step(s, hist, lens)
        kept += n_new
    assert max(kept) >= 3 and sum(kept) > 6 * N                 # drafts were accepted


def test_the_step_as_a_graph():
    dsa = lib()
    s, rng = Server(dsa), random.Random(6)
    hist, last = [[] for _ in range(N)], [1, 2, 3, 4, 5]
    s.draft(rng, last)                                          # (also loads what capturing may not)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.forward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        s.forward()
        s.keep()
    graph = {k: getattr(s, k) for k in ("pos", "q_raw", "kv_raw", "q", "kv", "logits")}
    for _ in range(4):
        lens = s.lens.tolist()
        s.draft(rng, last)                                      # (leaves its own tensors behind)
        for k, v in graph.items():
            setattr(s, k, v)
        g.replay()
        torch.cuda.synchronize()
        _, last = check_step(s, hist, lens)
