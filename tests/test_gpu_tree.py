"""Attention of drafted tokens over a paged cache against the fp64 definition.

Bounds.  bf16 path: P is rounded to bf16 (relative 2^-8 each at most), out is
rounded to bf16 (2^-8), and the logits are fp32 sums of 576 exact products: an
error of at most D = 576 * 2^-24 * S, S = max_s scale * sum_d |q_d k_d|, which
changes every weight exp(x - m) / l by a factor within exp(+-2 D); 2^-16 covers
ex2's error, the scaling's rounding and the fp32 sums over keys.  Hence
  |out - ref| <= (2^-8 + 2 * 2 D + 2^-16) * A + 2^-8 |ref|,  A = sum p |v| / l,
  |m - ref|   <= D + 2^-22 |ref| + 2^-22,    |l - ref| <= (2 D + 2^-16) ref.
fp32 path: the same with d_qk terms and without the two bf16 roundings (the sum
over n keys of fp32 terms: n * 2^-24 on top).
"""
import math
import random

import pytest
import torch

from gpu_util import DEV, lib
from oracle.tree import tree_attn

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Case:
    """Random cache and drafts; pages in random order, unused pool rows NaN."""

    def __init__(self, lens, T, H, R=64, kind="chain", d_qk=576, d_v=512, dtype=torch.bfloat16, seed=0, extra_tok=0,
                 q_scale=1.0):
        rng = random.Random(seed)
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        n = len(lens)
        T = [T] * n if isinstance(T, int) else T
        self.lens, self.T, self.H, self.R, self.d_qk, self.d_v, self.dtype = lens, T, H, R, d_qk, d_v, dtype
        pages = [-(-x // R) for x in lens]
        P, self.M = max(1, sum(pages)) + 3, max(1, max(pages))
        ids = list(range(P))
        rng.shuffle(ids)
        self.table, at = [], 0
        pool = torch.full((P, R, d_qk), math.nan, device=DEV)
        sc = 1.0 if dtype == torch.bfloat16 else d_qk ** -0.5
        for x, p in zip(lens, pages):
            row = ids[at:at + p]
            at += p
            self.table.append(row + [rng.choice([-1, 7 * P, 0])] * (self.M - p))
            if x:
                pos = torch.arange(x, device=DEV)
                pg = torch.tensor(row, device=DEV)[pos // R]
                pool[pg, pos % R] = torch.randn(x, d_qk, device=DEV, generator=gen) * sc
        self.pool = pool.to(dtype)
        self.tok_start = [0]
        for t in T:
            self.tok_start.append(self.tok_start[-1] + t)
        self.n_tok = max(1, self.tok_start[-1] + extra_tok)
        self.q = (torch.randn(self.n_tok, H, d_qk, device=DEV, generator=gen) * sc * q_scale).to(dtype)
        self.kv = (torch.randn(self.n_tok, d_qk, device=DEV, generator=gen) * sc).to(dtype)
        self.mask, self.words = None, 0
        if kind != "chain":
            self.words = max(1, -(-max(T) // 64)) + (1 if kind == "wide" else 0)
            rows = []
            for t in T:
                seen = []
                for i in range(t):
                    m = 1 << i
                    if kind == "tree" and i and rng.random() > 0.1:
                        m |= seen[rng.randrange(i)]
                    elif kind in ("any", "wide"):   # any set of drafted tokens, none among them
                        m = rng.getrandbits(t) & rng.getrandbits(t) if rng.random() > 0.2 else 0
                    elif kind == "none":
                        m = 0
                    seen.append(m)
                rows += seen
            rows += [(1 << 64 * self.words) - 1] * (self.n_tok - len(rows))
            w = [[(m >> (64 * k)) & ((1 << 64) - 1) for k in range(self.words)] for m in rows]
            self.mask = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in w], dtype=torch.int64,
                                     device=DEV)
        self.out = torch.full((self.n_tok, H, d_v), 7.0, dtype=dtype, device=DEV)
        self.m = torch.full((self.n_tok, H), 7.0, device=DEV)
        self.l = torch.full((self.n_tok, H), 7.0, device=DEV)

    def args(self, dsa):
        c = dsa.make_cache(n_seqs=len(self.lens), n_pages=self.pool.shape[0], page_rows=self.R, max_pages=self.M)
        t = dsa.make_tree(n_tok=self.n_tok, H=self.H, d_qk=self.d_qk, d_v=self.d_v, scale=SCALE,
                          dtype="bf16" if self.dtype == torch.bfloat16 else "fp32", mask_words=self.words)
        ws = torch.empty(max(16, dsa.tree_workspace_size(c, t)), dtype=torch.uint8, device=DEV).fill_(0xFF)
        return [c, t, self.q, self.pool, ints(self.table), ints(self.lens), self.kv, ints(self.tok_start), self.mask,
                self.out, self.m, self.l, ws]

    def run(self, dsa, status=0, **kw):
        dsa.tree_attn_fwd(*self.args(dsa), **kw)
        torch.cuda.synchronize()
        assert dsa.get_status() == status
        return self

    def reference(self):
        mask = None if self.mask is None else self.mask.cpu()
        scale = float(torch.tensor(SCALE, dtype=torch.float32))
        return tree_attn(self.q, self.pool, self.table, self.lens, self.kv, self.tok_start, mask, scale, self.d_v)

    def check(self, ref=None):
        out, m, l, A, S = ref or self.reference()
        n = self.tok_start[-1]
        bf = self.dtype == torch.bfloat16
        D = (self.d_qk * 2.0 ** -24 * S)[:n]
        more = 2.0 ** -16 if bf else 2.0 ** -20 + (max(self.lens) + max(self.T)) * 2.0 ** -24
        half = 2.0 ** -8 if bf else 2.0 ** -24
        for name, got, want, tol in (
                ("out", self.out[:n], out[:n], (half + 4 * D + more)[..., None] * A[:n] + half * out[:n].abs()),
                ("m", self.m[:n], m[:n], D + 2.0 ** -22 * m[:n].abs() + 2.0 ** -22),
                ("l", self.l[:n], l[:n], (2 * D + more) * l[:n])):
            got = got.double()
            fin = torch.isfinite(want)
            assert torch.equal(torch.isnan(got), torch.isnan(want)), name
            assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), name
            over = ((got - want).abs() - tol)[fin]
            assert over.numel() == 0 or float(over.max()) <= 0, (name, float((got - want).abs()[fin].max()))
        # what belongs to no sequence stays as it was
        assert (self.out[n:] == 7).all() and (self.m[n:] == 7).all() and (self.l[n:] == 7).all()
        return self


# cached lengths around blocks (112), boxes (16) and pages; heads that fill a tile,
# share it with other tokens, straddle it
BF16 = [
    ([0], 1, 128, 64, "chain"), ([1], 1, 128, 64, "chain"), ([15, 16, 17], 1, 128, 16, "chain"),
    ([111, 112, 113], 1, 16, 16, "chain"), ([1000], 1, 1, 64, "chain"), ([448, 447, 449], 1, 64, 112, "chain"),
    ([300, 0, 5], [3, 1, 2], 128, 48, "chain"), ([300, 0, 5, 77], [3, 0, 9, 1], 24, 64, "chain"),
    ([200, 33], [130, 1], 3, 64, "chain"), ([40], 230, 8, 16, "chain"), ([0, 0], [113, 112], 128, 16, "chain"),
    ([257, 1024], [12, 64], 128, 64, "tree"), ([257, 64], [12, 65], 16, 256, "tree"),
    ([100, 0], [64, 70], 5, 64, "any"), ([0, 3], [150, 20], 24, 32, "wide"), ([0, 700], [3, 2], 128, 64, "none"),
    ([9], 4, 200, 16, "any"), ([5000, 12000, 1], [2, 1, 5], 16, 64, "chain"), ([20000], 1, 128, 64, "chain"),
    ([3000] * 9, 1, 128, 64, "chain"),
]


@pytest.mark.parametrize("lens,T,H,R,kind", BF16)
def test_bf16(lens, T, H, R, kind):
    Case(lens, T, H, R, kind, extra_tok=3).run(lib()).check()


@pytest.mark.parametrize("lens,T,H,R,kind,d_qk,d_v", [
    ([0, 1, 127, 128, 129], 1, 3, 1, "chain", 80, 64), ([50, 0, 300], [5, 2, 0], 8, 24, "tree", 80, 64),
    ([10], 140, 2, 7, "any", 33, 17), ([3, 200], 2, 1, 16, "none", 1024, 1024), ([20, 0], [3, 70], 12, 5, "wide", 7, 7),
    ([64], 1, 1, 64, "chain", 1, 1)])
def test_fp32(lens, T, H, R, kind, d_qk, d_v):
    Case(lens, T, H, R, kind, d_qk, d_v, torch.float32, extra_tok=2).run(lib()).check()


def test_large_logits_move_the_maximum():
    # logits over hundreds: the running maximum rises often, O is rescaled, early weights vanish
    c = Case([900, 40], [2, 3], 64, 64, "tree", q_scale=30.0)
    c.pool[...] *= torch.linspace(0.1, 1.0, c.pool.shape[0], device=DEV).to(c.dtype)[:, None, None]
    c.run(lib()).check()


def test_batch_of_many_short_sequences():
    rng = random.Random(2)
    lens = [rng.choice([0, 1, 30, 200]) for _ in range(300)]
    T = [rng.choice([0, 1, 1, 2]) for _ in lens]
    Case(lens, T, 16, 16, "chain", extra_tok=1).run(lib()).check()


def test_same_bits_on_every_run():
    dsa = lib()
    c = Case([2000, 333], [5, 9], 64, 64, "tree").run(dsa)
    first = [x.clone() for x in (c.out, c.m, c.l)]
    c.run(dsa)
    assert all(torch.equal(a, b) for a, b in zip(first, (c.out, c.m, c.l)))


@pytest.mark.parametrize("H,dtype", [(128, torch.bfloat16), (16, torch.bfloat16), (4, torch.float32)])
def test_unseen_values_have_no_effect(H, dtype):
    # infinities and NaN in drafted rows: the tokens that see them get NaN, the
    # others exactly what they get without them
    dsa = lib()
    kw = dict(d_qk=576, d_v=512) if dtype == torch.bfloat16 else dict(d_qk=80, d_v=64)
    c = Case([130, 7], [40, 30], H, 16, "tree", dtype=dtype, **kw).run(dsa).check()
    clean = [x.clone() for x in (c.out, c.m, c.l)]
    # in value columns of either half and in the rope columns
    hit = {3: (5, math.nan), 17: (c.d_v - 1, math.nan), 45: (c.d_qk - 1, math.nan), 60: (c.d_v // 2, math.inf),
           33: (c.d_qk - 2, -math.inf), 52: (0, -math.inf)}
    for r, (col, v) in hit.items():
        c.kv[r, col] = v
    c.run(dsa)
    sees, nans = torch.zeros(70, dtype=torch.bool), torch.zeros(70, dtype=torch.bool)
    for r in range(70):
        t0 = 0 if r < 40 else 40
        bits = int(c.mask[r, 0])
        mine = [k for k in hit if t0 <= k < t0 + (40, 30)[t0 > 0] and (bits >> (k - t0)) & 1]
        sees[r], nans[r] = bool(mine), any(math.isnan(hit[k][1]) for k in mine)
    assert 0 < int(sees.sum()) < 70 and 0 < int(nans.sum())
    for got, was in zip((c.out, c.m, c.l), clean):
        assert torch.equal(got[~sees], was[~sees])
    assert torch.isnan(c.l[nans]).all() and torch.isnan(c.out[nans]).all()


def test_values_of_the_query_stay_in_their_row():
    dsa = lib()
    c = Case([300], 3, 16, 64, "chain").run(dsa)
    was = [x.clone() for x in (c.out, c.m, c.l)]
    c.q[1, 5, 100] = math.nan
    c.run(dsa)
    keep = torch.ones(3, 16, dtype=torch.bool)
    keep[1, 5] = False
    for got, w in zip((c.out, c.m, c.l), was):
        assert torch.equal(got[keep], w[keep])
    assert torch.isnan(c.out[1, 5]).all() and torch.isnan(c.l[1, 5])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_out_of_range_count_as_unseen(dtype):
    dsa = lib()
    kw = dict(d_qk=576, d_v=512) if dtype == torch.bfloat16 else dict(d_qk=80, d_v=64)
    c = Case([300, 100, 40], [2, 1, 1], 16, 16, "chain", dtype=dtype, **kw)
    c.table[0][3], c.table[0][18], c.table[1][0] = -1, c.pool.shape[0], 2 ** 31 - 1
    c.table[2] = [-5] * c.M
    c.run(dsa, status=dsa.DSA_ERR_INDEX).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sequences_out_of_range_are_left_out(dtype):
    dsa = lib()
    kw = dict(d_qk=576, d_v=512) if dtype == torch.bfloat16 else dict(d_qk=80, d_v=64)
    c = Case([100, 50, 30], [2, 3, 70], 8, 16, "tree", dtype=dtype, **kw)
    good = Case([100, 50, 30], [2, 3, 70], 8, 16, "tree", dtype=dtype, **kw).run(dsa)
    c.lens = [100, c.M * 16 + 1, -1]
    c.run(dsa, status=dsa.DSA_ERR_INDEX)
    assert torch.equal(c.out[:2], good.out[:2]) and (c.out[2:] == 7).all() and (c.l[2:] == 7).all()
    c.lens, c.words, c.mask = [100, 50, 30], 1, c.mask[:, :1].contiguous()   # 70 tokens, 64 mask bits
    c.run(dsa, status=dsa.DSA_ERR_INDEX)
    assert torch.equal(c.out[:5], good.out[:5]) and (c.out[5:] == 7).all()


def test_pool_of_interleaved_layers():
    dsa = lib()
    c = Case([500, 37], [2, 3], 32, 32, "chain")
    layers = torch.randn(c.pool.shape[0], 3, 32, 576, device=DEV).to(torch.bfloat16)
    layers[:, 1] = c.pool
    want = c.run(dsa).out.clone()
    c.pool = layers[:, 1]
    c.out.fill_(7)
    assert torch.equal(c.run(dsa).out, want)


def test_pool_past_four_gigabytes():
    dsa = lib()
    c = Case([400, 65], 2, 16, 64, "chain")
    want = c.run(dsa).out.clone()
    far = torch.zeros(70000, 64, 576, dtype=torch.bfloat16, device=DEV)
    for row in c.table:
        for j, p in enumerate(row):
            if 0 <= p < c.pool.shape[0]:
                far[69990 - p] = c.pool[p]
                row[j] = 69990 - p
    c.pool = far
    c.out.fill_(7)
    assert torch.equal(c.run(dsa).out, want)


def test_other_streams_and_graphs_with_new_lengths():
    dsa = lib()
    big = Case([900, 1200, 700], [3, 2, 4], 64, 64, "chain")
    a = big.args(dsa)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dsa.tree_attn_fwd(*a, stream=side)
    torch.cuda.synchronize()
    big.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        dsa.tree_attn_fwd(*a)
    for lens, starts in (([900, 0, 33], [0, 3, 5, 9]), ([1, 1200, 699], [0, 1, 1, 9]), ([64, 64, 64], [0, 9, 9, 9])):
        big.lens, big.tok_start = lens, starts
        big.T = [y - x for x, y in zip(starts, starts[1:])]
        a[5].copy_(ints(lens))
        a[7].copy_(ints(starts))
        for x in (big.out, big.m, big.l):
            x.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert dsa.get_status() == 0
        big.check()


def test_agrees_with_the_sparse_attention_that_keeps_every_key():
    # one prompt chunk: the selection of every cached and earlier drafted key
    dsa = lib()
    n, T, H = 200, 9, 128
    c = Case([n], T, H, 16, "chain").run(dsa)
    pos = torch.arange(n, device=DEV)
    kv = torch.cat([c.pool[torch.tensor(c.table[0], device=DEV)[pos // 16], pos % 16], c.kv])[None].contiguous()
    k = 256
    p = dsa.make_params(B=1, S_q=T, S_k=n + T, H=H, d_qk=576, d_v=512, H_I=64, d_I=128, topk=k, scale=SCALE,
                        q_row_offset=n)
    idx = torch.full((1, T, k), -1, dtype=torch.int32, device=DEV)
    for t in range(T):
        idx[0, t, :n + t + 1] = torch.arange(n + t + 1, device=DEV)
    out = torch.empty(1, T, H, 512, dtype=torch.bfloat16, device=DEV)
    m, l = torch.empty(1, T, H, device=DEV), torch.empty(1, T, H, device=DEV)
    dsa.sparse_attn_fwd(p, c.q[None].contiguous(), kv, idx, out, m, l)
    torch.cuda.synchronize()
    c.check()
    ref = c.reference()
    c.out, c.m, c.l = out[0], m[0], l[0]
    c.check(ref)


def test_refused_calls():
    dsa = lib()
    c = Case([40], 2, 8, 16, "tree")
    base = c.args(dsa)

    def refused(code, **kw):
        a = list(base)
        for k, v in kw.items():
            a[dict(cache=0, tree=1, q=2, pool=3, mask=8, ws=12)[k]] = v
        with pytest.raises(dsa.DSAError) as e:
            dsa.tree_attn_fwd(*a)
        assert e.value.code == code

    mk = lambda **kw: dsa.make_tree(**dict(dict(n_tok=2, H=8, d_qk=576, d_v=512, scale=SCALE, mask_words=1), **kw))
    refused(dsa.DSA_ERR_INVALID_ARG, mask=None)                       # mask words, no mask
    refused(dsa.DSA_ERR_INVALID_ARG, tree=mk(scale=0.0))
    refused(dsa.DSA_ERR_WORKSPACE, ws=None)
    refused(dsa.DSA_ERR_WORKSPACE, ws=base[12][:-16])
    off = torch.empty(c.pool.numel() + 4, dtype=torch.bfloat16, device=DEV)[4:].view_as(c.pool)
    refused(dsa.DSA_ERR_INVALID_ARG, pool=off)                        # not 16-byte aligned
    odd = dsa.make_cache(n_seqs=1, n_pages=4, page_rows=24, max_pages=c.M)
    with pytest.raises(dsa.DSAError) as e:
        dsa.tree_attn_fwd(odd, base[1], c.q, torch.zeros(4, 24, 576, dtype=torch.bfloat16, device=DEV), *base[4:])
    assert e.value.code == dsa.DSA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        dsa.tree_attn_fwd(base[0], base[1], c.q[:1], *base[3:])
    with pytest.raises(TypeError):
        dsa.tree_attn_fwd(base[0], base[1], c.q.half(), *base[3:])


@pytest.mark.parametrize("H,T", [(4, [3, 1, 2]), (4, [40, 21, 39]), (9, [30, 20, 34])])
def test_fp32_with_keys_shared_by_four_two_and_one_cta(H, T):
    dsa = lib()
    Case([701, 0, 130], T, H, R=16, kind="any", d_qk=80, d_v=64, dtype=torch.float32, seed=H).run(dsa).check()
    Case([1500, 40, 129], T, H, R=1, d_qk=33, d_v=7, dtype=torch.float32, seed=H + 1).run(dsa).check()


@pytest.mark.parametrize("H,T,R,kind", [(128, 1, 64, "chain"), (16, 9, 32, "tree"), (128, 3, 96, "any")])
def test_bad_pages_between_full_blocks(H, T, R, kind):
    dsa = lib()
    c = Case([2000, 5000, 111], T, H, R=R, kind=kind, seed=R)
    for i, js in ((0, (0, 7)), (1, (3, 20, 21, 4999 // R))):
        for j in js:
            c.table[i][j] = (-3, c.pool.shape[0])[j % 2]
    c.run(dsa, status=dsa.DSA_ERR_INDEX).check()


@pytest.mark.parametrize("lens,T,H,kind", [
    ([336, 448, 560], 40, 128, "tree"), ([224] * 30, 9, 128, "chain"), ([230] * 40, 5, 128, "any"),
    ([3360], 100, 128, "chain")])
def test_every_block_of_every_tile_moves_the_maximum(lens, T, H, kind):
    # logits rise by 9 from one block of 112 keys to the next (more than O may lag behind, 8 ln 2): short
    # tiles one after the other, O rescaled in each of their cached blocks
    dsa = lib()
    c = Case(lens, T, H, 64, kind)
    u = torch.randn(c.d_qk, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5))
    u *= SCALE ** -0.5 / u.norm()
    c.q = (c.q.float() * 0.25 + u).to(c.dtype)
    for b, n in enumerate(lens):
        pos = torch.arange(n, device=DEV)
        pg = torch.tensor(c.table[b], device=DEV)[pos // c.R]
        c.pool[pg, pos % c.R] = (c.pool[pg, pos % c.R].float() * 0.25 + (pos // 112)[:, None] * 9.0 * u).to(c.dtype)
    c.run(dsa).check()
    first = [x.clone() for x in (c.out, c.m, c.l)]
    for _ in range(20):
        c.out.fill_(7)
        c.run(dsa)
        assert all(torch.equal(a, b) for a, b in zip(first, (c.out, c.m, c.l)))


@pytest.mark.parametrize("lens,T,H,kind,dtype", [
    ([700], 1500, 16, "chain", torch.bfloat16), ([0, 130, 2001], [900, 0, 513], 24, "chain", torch.bfloat16),
    ([300], 700, 128, "chain", torch.bfloat16), ([50, 513], [1000, 300], 8, "tree", torch.bfloat16),
    ([0, 90], [700, 129], 5, "chain", torch.float32), ([200], 400, 6, "any", torch.float32)])
def test_chunk_of_a_prompt(lens, T, H, kind, dtype):
    # more drafted rows than cached ones, over many blocks and words of mask bits
    kw = dict(d_qk=576, d_v=512) if dtype == torch.bfloat16 else dict(d_qk=80, d_v=64)
    Case(lens, T, H, 64, kind, dtype=dtype, extra_tok=2, **kw).run(lib()).check()


def test_calls_on_two_streams_at_once():
    # each with a workspace of its own
    dsa = lib()
    cases = [Case([900, 3000, 40], [3, 2, 40], 64, 64, "tree", seed=1), Case([5000], 9, 128, 64, "chain", seed=2)]
    args = [c.args(dsa) for c in cases]
    want = []
    for c, a in zip(cases, args):
        dsa.tree_attn_fwd(*a)
        torch.cuda.synchronize()
        c.check()
        want.append([x.clone() for x in (c.out, c.m, c.l)])
        for x in (c.out, c.m, c.l):
            x.fill_(7)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for a, s in zip(args, streams):
            dsa.tree_attn_fwd(*a, stream=s)
    torch.cuda.synchronize()
    assert dsa.get_status() == 0
    for c, w in zip(cases, want):
        assert all(torch.equal(x, y) for x, y in zip((c.out, c.m, c.l), w))
