"""The decoding calls together, as a server makes them: a beam search and a run of
accepted drafts, eagerly and as a replayed graph.

Each sequence's cache must hold, bit for bit, the rows of that sequence's own
tokens after any number of forks, extensions, writes and compactions; the
attention is compared with the fp64 definition over those rows (bounds as in
test_gpu_tree), the selection with the definition over the logits it was given.
"""
import math
import random

import pytest
import torch

from gpu_util import DEV, lib
from oracle.beam import beam_select
from oracle.tree import tree_attn

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
D, DV = 576, 512


def ints(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device=DEV)


class Cache:
    """A cache with a latent pool and a two-layer pool of odd rows; two tables that take turns through a copy."""

    def __init__(self, dsa, n, P, R, M, n_slots):
        self.dsa, self.c = dsa, dsa.make_cache(n_seqs=n, n_pages=P, page_rows=R, max_pages=M)
        self.n, self.P, self.R, self.M = n, P, R, M
        self.pool = torch.full((P, R, D), math.nan, dtype=torch.bfloat16, device=DEV)
        self.keys = torch.zeros((2, P, R, 133), dtype=torch.uint8, device=DEV)
        self.table, self.lens, self.refs = ints(n, M, fill=-1), ints(n), ints(P)
        self.out = ints(n, M), ints(n), ints(P)
        self.map = ints(P)
        self.copies, self.n_copies = ints(max(n, P // 2 + 1), 3), ints(1)
        self.slots = ints(n_slots)

    def moved(self, with_lens):
        for pool in (self.pool, self.keys):
            self.dsa.cache_copy_pages(self.c, pool, self.copies, self.n_copies)
        self.table.copy_(self.out[0])
        self.refs.copy_(self.out[2])
        if with_lens:
            self.lens.copy_(self.out[1])

    def fork(self, parent):
        self.dsa.cache_fork(self.c, parent, self.table, self.lens, self.refs, *self.out, self.copies, self.n_copies)
        self.moved(True)

    def compact(self):
        self.dsa.cache_compact(self.c, self.table, self.lens, self.refs, self.out[0], self.out[2], self.map,
                               self.copies, self.n_copies)
        self.moved(False)

    def append(self, n_new, rows, keys, row_index=None):
        self.dsa.cache_extend(self.c, n_new, self.table, self.lens, self.refs, self.lens, self.refs, self.slots)
        self.dsa.cache_write(self.c, self.pool, rows, self.slots, row_index)
        self.dsa.cache_write(self.c, self.keys, keys, self.slots, row_index)

    def check(self, hist, kv, keys):
        """Sequence i holds the rows of tokens hist[i], each page as often as refs says."""
        table, lens, refs = self.table.tolist(), self.lens.tolist(), self.refs.tolist()
        assert lens == [len(h) for h in hist]
        uses = [0] * self.P
        for i, h in enumerate(hist):
            pages = table[i][:-(-len(h) // self.R)]
            for p in pages:
                uses[p] += 1
            if h:
                rows = torch.tensor([pages[x // self.R] * self.R + x % self.R for x in range(len(h))], device=DEV)
                assert torch.equal(self.pool.view(-1, D)[rows].view(torch.int16), kv[h].view(torch.int16))
                assert torch.equal(self.keys.view(2, -1, 133)[:, rows], keys[:, h])
        assert uses == refs


def check_attn(got, q, hist, kv, kv_new, tok_start, mask):
    """out of every drafted token against the definition over the sequences' own rows."""
    longest = max(1, max(len(h) for h in hist))
    pool = torch.zeros((len(hist), longest, D), dtype=torch.bfloat16, device=DEV)
    for i, h in enumerate(hist):
        if h:
            pool[i, :len(h)] = kv[h]
    scale = float(torch.tensor(SCALE, dtype=torch.float32))
    out, _, _, A, S = tree_attn(q, pool, [[i] for i in range(len(hist))], [len(h) for h in hist], kv_new, tok_start,
                                mask, scale, DV)
    n = tok_start[-1]
    tol = (2.0 ** -8 + 4 * D * 2.0 ** -24 * S[:n] + 2.0 ** -16)[..., None] * A[:n] + 2.0 ** -8 * out[:n].abs()
    assert bool(((got[:n].double() - out[:n]).abs() <= tol).all())


def stepper(step, graph):
    """step itself, or its replay: captured after one eager run on a side stream (the state must be reset after)."""
    if not graph:
        return step
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    return g.replay


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("n_batch,W,V,H,R,steps", [(2, 3, 40, 4, 16, 40), (1, 5, 512, 16, 32, 70), (3, 1, 100, 128, 64, 5)])
def test_beam_search(n_batch, W, V, H, R, steps, graph):
    dsa = lib()
    n, M = n_batch * W, -(-steps // R)
    gen = torch.Generator(device=DEV).manual_seed(n + V)
    eos = 3
    kv = torch.randn(V, D, device=DEV, generator=gen).to(torch.bfloat16)
    keys = torch.randint(0, 256, (2, V, 133), dtype=torch.uint8, device=DEV, generator=gen)
    emb = torch.randn(V, H, D, device=DEV, generator=gen).to(torch.bfloat16)
    noise = torch.randn(steps + 2, n, V, device=DEV, generator=gen)
    cache = Cache(dsa, n, n * M + 1, R, M, n)
    t = dsa.make_tree(n_tok=n, H=H, d_qk=D, d_v=DV, scale=SCALE)
    b = dsa.make_beam(n_batch=n_batch, beams_in=W, beams_out=W, vocab=V, dtype="fp32", eos=eos)
    ws_t = torch.empty(dsa.tree_workspace_size(cache.c, t), dtype=torch.uint8, device=DEV)
    ws_b = torch.empty(dsa.beam_workspace_size(b), dtype=torch.uint8, device=DEV)
    ones, start = ints(n, fill=1), torch.arange(n + 1, dtype=torch.int32, device=DEV)
    out = torch.empty(n, H, DV, dtype=torch.bfloat16, device=DEV)
    m, l = torch.empty(n, H, device=DEV), torch.empty(n, H, device=DEV)
    tok, parent, at = ints(n, fill=1), ints(n), torch.zeros(1, dtype=torch.int64, device=DEV)
    score, fin = torch.zeros(n, device=DEV), torch.zeros(n, dtype=torch.uint8, device=DEV)
    score_out, fin_out = torch.empty_like(score), torch.empty_like(fin)
    logits, q = torch.empty(n, V, device=DEV), torch.empty(n, H, D, dtype=torch.bfloat16, device=DEV)
    rows, row_keys = torch.empty(n, D, dtype=torch.bfloat16, device=DEV), torch.empty(2, n, 133, dtype=torch.uint8, device=DEV)
    score_in, fin_in = torch.empty_like(score), torch.empty_like(fin)

    def step():
        score_in.copy_(score), fin_in.copy_(fin)
        q.copy_(emb[tok.long()]), rows.copy_(kv[tok.long()]), row_keys.copy_(keys[:, tok.long()])
        dsa.tree_attn_fwd(cache.c, t, q, cache.pool, cache.table, cache.lens, rows, start, None, out, m, l, ws_t)
        logits.copy_(2 * out[:, 0, :V].float() + noise[at].squeeze(0))
        cache.append(ones, rows, row_keys)
        dsa.beam_select(b, logits, score, fin, parent, tok, score_out, fin_out, ws_b)
        cache.fork(parent)
        score.copy_(score_out), fin.copy_(fin_out), at.add_(1)

    run = stepper(step, graph)
    for x in (cache.lens, cache.refs, fin, at):
        x.zero_()
    tok.fill_(1)
    score.copy_(torch.tensor(([0.0] + [-math.inf] * (W - 1)) * n_batch))
    hist, now = [[] for _ in range(n)], [1] * n
    for k in range(steps):
        run()
        torch.cuda.synchronize()
        assert dsa.get_status() == 0
        if k < 3 or k % 8 == 0:
            check_attn(out, q, hist, kv, rows, start.tolist(), None)
        want = beam_select(logits.view(n_batch, W, V).double().tolist(), score_in.view(n_batch, W).tolist(),
                           fin_in.view(n_batch, W).tolist(), W, eos)
        want = [x for r in want for x in r]
        assert parent.tolist() == [x[0] for x in want] and tok.tolist() == [x[1] for x in want]
        assert [bool(x) for x in fin.tolist()] == [x[3] for x in want]
        grown = [h + [x] for h, x in zip(hist, now)]
        hist, now = [list(grown[x[0]]) for x in want], [x[1] for x in want]
        cache.check(hist, kv, keys)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("n,T,H,R", [(3, 5, 4, 16), (2, 17, 16, 48), (1, 64, 128, 64)])
def test_draft_and_accept(n, T, H, R, graph):
    dsa = lib()
    steps, V = 7, 30
    rng = random.Random(n * T)
    gen = torch.Generator(device=DEV).manual_seed(T)
    M = -(-(steps + 1) * T // R)
    kv = torch.randn(V, D, device=DEV, generator=gen).to(torch.bfloat16)
    keys = torch.randint(0, 256, (2, V, 133), dtype=torch.uint8, device=DEV, generator=gen)
    cache = Cache(dsa, n, n * M + 2, R, M, n * T)
    t = dsa.make_tree(n_tok=n * T, H=H, d_qk=D, d_v=DV, scale=SCALE, mask_words=1)
    ws = torch.empty(dsa.tree_workspace_size(cache.c, t), dtype=torch.uint8, device=DEV)
    q = torch.randn(n * T, H, D, device=DEV, generator=gen).to(torch.bfloat16)
    out = torch.empty(n * T, H, DV, dtype=torch.bfloat16, device=DEV)
    m, l = torch.empty(n * T, H, device=DEV), torch.empty(n * T, H, device=DEV)
    start = torch.arange(0, n * T + 1, T, dtype=torch.int32, device=DEV)
    tok, mask = torch.zeros(n * T, dtype=torch.int64, device=DEV), torch.zeros(n * T, 1, dtype=torch.int64, device=DEV)
    n_new, accepted, parent = ints(n), ints(n * T), torch.arange(n, dtype=torch.int32, device=DEV)
    rows = torch.empty(n * T, D, dtype=torch.bfloat16, device=DEV)

    def step():
        rows.copy_(kv[tok])
        dsa.tree_attn_fwd(cache.c, t, q, cache.pool, cache.table, cache.lens, rows, start, mask, out, m, l, ws)
        cache.append(n_new, rows, keys[:, tok].contiguous(), accepted)
        cache.fork(parent)
        cache.compact()

    run = stepper(step, graph)
    cache.lens.zero_(), cache.refs.zero_()
    hist = [[] for _ in range(n)]
    for k in range(steps):
        toks = [rng.randrange(V) for _ in range(n * T)]
        masks, paths = [], []
        for i in range(n):
            up = []                                # a random tree; a path from its root is accepted
            for j in range(T):
                up.append(rng.randrange(-1, j) if j else -1)
                masks.append((1 << j) | (masks[i * T + up[j]] if up[j] >= 0 else 0))
            path, j = [], rng.randrange(T) if rng.random() < 0.8 else -1
            while j >= 0:
                path.append(i * T + j)
                j = up[j]
            paths.append(path[::-1])
        # the last step but one empties a sequence, the one before makes all of them copies of one
        par = [0] * n if k == steps - 3 else [-1] + list(range(1, n)) if k == steps - 2 else list(range(n))
        flat = [x for p in paths for x in p]
        tok.copy_(torch.tensor(toks))
        mask.copy_(torch.tensor([[x - (1 << 64) if x >> 63 else x] for x in masks]))
        n_new.copy_(torch.tensor([len(p) for p in paths], dtype=torch.int32))
        accepted.copy_(torch.tensor(flat + [0] * (n * T - len(flat)), dtype=torch.int32))
        parent.copy_(torch.tensor(par, dtype=torch.int32))
        run()
        torch.cuda.synchronize()
        assert dsa.get_status() == 0
        check_attn(out, q, hist, kv, rows, start.tolist(), mask.cpu())
        grown = [h + [toks[x] for x in p] for h, p in zip(hist, paths)]
        hist = [list(grown[p]) if p >= 0 else [] for p in par]
        cache.check(hist, kv, keys)
        held = sum(r > 0 for r in cache.refs.tolist())
        assert all(r > 0 for r in cache.refs.tolist()[:held])


def test_native_marshalling_is_there_and_python_agrees(monkeypatch):
    """The calls go through the compiled module; without it the same functions give the same steps."""
    dsa = lib()
    assert hasattr(dsa._native, "bind")
    answers = []

    class Spy:
        def __getattr__(self, name):
            def call(*args):
                answers.append((name, getattr(native, name)(*args)))
                return answers[-1][1]
            return call

    native = dsa._native
    monkeypatch.setattr(dsa, "_native", Spy())
    test_beam_search(1, 2, 20, 3, 16, 18, False)
    test_draft_and_accept(2, 5, 4, 16, False)
    assert {n for n, _ in answers} == {"cache_fork", "cache_extend", "cache_compact", "cache_copy_pages", "cache_write",
                                       "tree_attn_fwd", "beam_select"}
    assert all(a == 0 for _, a in answers)
    monkeypatch.setattr(dsa, "_native", dsa._Absent())
    test_beam_search(1, 2, 20, 3, 16, 18, False)
    test_draft_and_accept(2, 5, 4, 16, False)


def test_native_marshalling_refuses_what_the_python_code_refuses():
    dsa = lib()
    n, P, R, M = 2, 6, 16, 3
    c = dsa.make_cache(n_seqs=n, n_pages=P, page_rows=R, max_pages=M)
    good = dict(parent=ints(n), table=ints(n, M, fill=-1), lens=ints(n), refs=ints(P), table_out=ints(n, M),
                lens_out=ints(n), refs_out=ints(P), copies=ints(n, 3), n_copies=ints(1))
    fork = lambda c=c, **kw: dsa._native.cache_fork(c, *{**good, **kw}.values())
    assert fork() == 0
    bad = [dict(table=good["table"].cpu()), dict(lens=ints(n).long()), dict(refs=ints(P + 1)), dict(copies=ints(n, 2)),
           dict(table=ints(M, n).t()), dict(n_copies=None), dict(parent=[0, 0]), dict(lens_out=ints(2 * n)[::2])]
    for kw in bad:
        assert fork(**kw) == 1
        with pytest.raises((TypeError, ValueError)):
            dsa.cache_fork(c, *{**good, **kw}.values())
    assert fork(c=b"x" * 32) == 1 and fork(c=dsa.make_beam(n_batch=1, beams_in=1, beams_out=1, vocab=1)) == 1
    assert dsa._native.cache_fork(c) == 1
    wide = dsa.make_cache(n_seqs=2 ** 62, n_pages=P, page_rows=R, max_pages=2 ** 62)
    assert fork(c=wide) == 1
    # what the library itself refuses comes back as its error
    assert fork(table_out=good["table"]) == dsa.DSA_ERR_INVALID_ARG
    with pytest.raises(dsa.DSAError):
        dsa.cache_fork(c, *{**good, "table_out": good["table"]}.values())
    # another stream than the current one, given or current
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dsa.cache_fork(c, *good.values(), stream=s)
    with torch.cuda.stream(s):
        assert fork() == 0
    torch.cuda.synchronize()
    assert dsa.get_status() == 0
