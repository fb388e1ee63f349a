"""Beam selection on the GPU against the fp64 definition.

Indices must be equal; inputs keep candidates of different beams apart (or make
them equal exactly).  Scores: a term exp(-d), d = max - x, has a relative error
of at most d 2^-23 (the roundings of d and of d log2 e) + 2^-22 (the
exponential's own 2 units), so the sum is off by the mean of that over the
softmax's weights.  The mean of d is below 5 for every input here (some 4.5
for the normal logits of deviation 2.5), which gives less than 2^-20 for the
logarithm, its own error of 2^-24 included; then the score is rounded to fp32.
"""
import math
import random

import pytest
import torch

from gpu_util import DEV, lib
from oracle.beam import beam_select

pytestmark = pytest.mark.gpu
INF = math.inf


def run(dsa, logits, scores, finished, keep, eos, ld=None, dtype=torch.float32, offset=0):
    """logits [n, W, V] (any float tensor) -> lists (parent, token, score, finished)."""
    n, W, V = logits.shape
    ld = ld or V
    store = torch.full((n * W * ld + offset,), INF, dtype=dtype, device=DEV)  # what lies between the rows is not read
    x = store[offset:].view(n, W, ld)
    x[..., :V] = logits.to(dtype)
    b = dsa.make_beam(n_batch=n, beams_in=W, beams_out=keep, vocab=V, ld=ld,
                      dtype="bf16" if dtype == torch.bfloat16 else "fp32", eos=eos)
    ws = torch.empty(dsa.beam_workspace_size(b), dtype=torch.uint8, device=DEV).fill_(0xA5)
    fin = None if finished is None else torch.tensor(finished, dtype=torch.uint8, device=DEV)
    o = [torch.full((n, keep), 7, dtype=t, device=DEV) for t in (torch.int32, torch.int32, torch.float32, torch.uint8)]
    dsa.beam_select(b, x, torch.tensor(scores, device=DEV, dtype=torch.float32), fin, *o, ws)
    torch.cuda.synchronize()
    assert dsa.get_status() == 0
    return [list(zip(*(t[i].tolist() for t in o))) for i in range(n)]


def check(dsa, logits, scores, finished, keep, eos, **kw):
    dtype = kw.get("dtype", torch.float32)
    got = run(dsa, logits, scores, finished, keep, eos, **kw)
    sc = torch.tensor(scores, dtype=torch.float32).tolist()
    want = beam_select(logits.to(dtype).double().tolist(), sc, finished, keep, eos)
    for g, w in zip(got, want):
        assert [(p, t, bool(f)) for p, t, _, f in g] == [(p, t, f) for p, t, _, f in w]
        for (_, _, a, _), (_, _, b, _) in zip(g, w):
            assert a == b or abs(a - b) <= 2.0 ** -20 + 2.0 ** -23 * abs(b)


def rand(*shape, seed=0, scale=2.5):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,W,V,keep,ld,offset", [
    (1, 1, 1, 1, None, 0), (1, 1, 5, 8, None, 0), (2, 3, 2, 6, 7, 0), (1, 4, 1000, 4, None, 0),
    (3, 2, 8191, 2, None, 1), (2, 2, 8192, 5, None, 0), (2, 2, 8193, 5, 8200, 0), (1, 5, 32001, 32, None, 3),
    (2, 32, 301, 32, 304, 0), (1, 2, 70000, 3, 70016, 0), (5, 8, 257, 8, None, 0)])
def test_random(n, W, V, keep, ld, offset, dtype):
    dsa = lib()
    scores = (-20 * torch.rand(n, W, generator=torch.Generator().manual_seed(V))).tolist()
    check(dsa, rand(n, W, V, seed=V + W), scores, None, keep, -1, ld=ld, dtype=dtype, offset=offset)
    rng = random.Random(V)
    fin = [[int(rng.random() < 0.4) for _ in range(W)] for _ in range(n)]
    dead = [[-INF if rng.random() < 0.3 else s for s in r] for r in scores]
    check(dsa, rand(n, W, V, seed=V), dead, fin, keep, rng.randrange(V), ld=ld, dtype=dtype, offset=offset)


def test_first_step_and_equal_beams():
    # one live beam; then beams with equal rows and equal scores: ties go to the lower beam,
    # whatever the rows' alignment
    dsa = lib()
    x = rand(1, 1, 1001, seed=3).expand(2, 4, 1001).contiguous()
    check(dsa, x, [[0.0, -INF, -INF, -INF]] * 2, None, 4, 0)
    for dtype in (torch.float32, torch.bfloat16):
        got = run(dsa, x, [[-1.5] * 4] * 2, None, 8, 0, dtype=dtype)
        best = run(dsa, x[:, :1], [[-1.5]] * 2, None, 2, 0, dtype=dtype)
        for b in range(2):
            assert [(p, t) for p, t, _, _ in got[b]] == \
                [(4 * b + w, best[b][i][1]) for i in range(2) for w in range(4)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_and_order_within_a_beam(dtype):
    dsa = lib()
    check(dsa, torch.zeros(2, 2, 20000, dtype=torch.float64), [[-1.0, -2.0]] * 2, None, 32, 5, dtype=dtype)
    x = (rand(1, 2, 30000, seed=9).round() * 0.5)                 # many equal logits
    check(dsa, x, [[-1.0, -30.0]], None, 32, 5, dtype=dtype)
    up = torch.arange(20000, dtype=torch.float64)[None, None] / 128   # the best are all in one thread's hands
    check(dsa, up, [[0.0]], None, 32, 19999, dtype=dtype)
    check(dsa, -up, [[0.0]], None, 32, 0, dtype=dtype)
    signed = torch.zeros(1, 1, 300, dtype=torch.float64)
    signed[..., ::2] = -0.0                                       # -0 and +0 are one value
    check(dsa, signed, [[0.0]], None, 10, 0, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_and_unusable_logits(dtype):
    dsa = lib()
    x = rand(2, 3, 9000, seed=4)
    x[0, 0, 10:] = -INF                      # fewer logits than are kept
    x[0, 1] = -INF                           # none
    x[0, 2, 5], x[0, 2, 6], x[0, 2, 8999] = INF, math.nan, -INF
    x[1, 0, :8192] = -INF                    # a whole chunk
    x[1, 1] = torch.finfo(dtype).min         # the type's lowest value is a logit like any other
    x[1, 2, ::2] = math.nan
    check(dsa, x, [[-1.0, 0.0, -40.0], [-1.0, -2.0, -3.0]], None, 16, -1, dtype=dtype)
    check(dsa, x[:1, :2].contiguous(), [[-1.0, 0.0]], None, 16, -1, dtype=dtype)
    check(dsa, x[:1, 1:2].contiguous(), [[-1.0]], None, 4, -1, dtype=dtype)


def test_large_spread():
    # logits far apart, scores far below
    dsa = lib()
    x = rand(2, 2, 5000, seed=6, scale=60.0)
    check(dsa, x, [[-1000.0, -1003.0], [0.0, -3.4e38]], None, 8, -1)


def test_graph_replay_on_new_logits_and_other_stream():
    dsa = lib()
    n, W, V, K = 3, 4, 9001, 4
    b = dsa.make_beam(n_batch=n, beams_in=W, beams_out=K, vocab=V, dtype="fp32", eos=2)
    ws = torch.empty(dsa.beam_workspace_size(b), dtype=torch.uint8, device=DEV)
    x, s = torch.zeros(n, W, V, device=DEV), torch.zeros(n, W, device=DEV)
    f = torch.zeros(n, W, dtype=torch.uint8, device=DEV)
    o = [torch.zeros(n, K, dtype=t, device=DEV) for t in (torch.int32, torch.int32, torch.float32, torch.uint8)]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        dsa.beam_select(b, x, s, f, *o, ws)
    for seed in range(3):
        y = rand(n, W, V, seed=seed)
        x.copy_(y)
        s.copy_(rand(n, W, seed=seed + 50))
        f.copy_(rand(n, W, seed=seed + 90) > 2)
        g.replay()
        torch.cuda.synchronize()
        want = beam_select(y.float().double().tolist(), s.tolist(), f.tolist(), K, 2)
        for i in range(n):
            assert [(p, t, bool(z)) for p, t, z in zip(o[0][i].tolist(), o[1][i].tolist(), o[3][i].tolist())] == \
                [(p, t, z) for p, t, _, z in want[i]]


def test_rows_past_four_gigabytes():
    dsa = lib()
    n, W, V, ld = 3, 3, 1000, 300_000_000
    store = torch.zeros(n * W * ld, dtype=torch.bfloat16, device=DEV)
    x = store.view(n, W, ld)
    y = rand(n, W, V, seed=1).to(torch.bfloat16)
    x[..., :V] = y.to(DEV)
    b = dsa.make_beam(n_batch=n, beams_in=W, beams_out=3, vocab=V, ld=ld, eos=-1)
    ws = torch.empty(dsa.beam_workspace_size(b), dtype=torch.uint8, device=DEV)
    o = [torch.zeros(n, 3, dtype=t, device=DEV) for t in (torch.int32, torch.int32, torch.float32)]
    s = torch.zeros(n, W, device=DEV)
    dsa.beam_select(b, x, s, None, *o, None, ws)
    want = beam_select(y.double().tolist(), s.tolist(), None, 3, -1)
    assert [list(zip(a, c)) for a, c in zip(o[0].tolist(), o[1].tolist())] == [[(p, t) for p, t, _, _ in r] for r in want]


def test_refused_calls():
    dsa = lib()
    x, s = torch.zeros(1, 2, 8, device=DEV), torch.zeros(1, 2, device=DEV)
    f = torch.zeros(1, 2, dtype=torch.uint8, device=DEV)
    o = [torch.zeros(1, 2, dtype=t, device=DEV) for t in (torch.int32, torch.int32, torch.float32, torch.uint8)]
    mk = lambda **kw: dsa.make_beam(**dict(dict(n_batch=1, beams_in=2, beams_out=2, vocab=8, dtype="fp32"), **kw))
    ws = torch.empty(dsa.beam_workspace_size(mk()), dtype=torch.uint8, device=DEV)
    with pytest.raises(dsa.DSAError) as e:   # finished beams need an end token
        dsa.beam_select(mk(), x, s, f, *o, ws)
    assert e.value.code == dsa.DSA_ERR_INVALID_ARG
    with pytest.raises(dsa.DSAError) as e:
        dsa.beam_select(mk(), x, s, None, *o, ws[:-1])
    assert e.value.code == dsa.DSA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        dsa.beam_select(mk(), x[..., :7], s, None, *o, ws)
    with pytest.raises(TypeError):
        dsa.beam_select(mk(dtype="bf16"), x, s, None, *o, ws)


@pytest.mark.parametrize("W,V,keep,dtype", [
    (1, 140001, 32, torch.float32), (2, 300000, 5, torch.float32), (1, 530001, 9, torch.float32),
    (1, 270001, 32, torch.bfloat16)])
def test_long_vocabularies(W, V, keep, dtype):
    """Rows of more chunks than a warp has lanes, and of more than its lanes have lists."""
    dsa = lib()
    x = rand(1, W, V, seed=V)
    x[0, 0, V - 40:] += 12.0                     # many of the best in the last chunk, some in others
    check(dsa, x, [[-1.5] * W], None, keep, -1, dtype=dtype)


def test_scores_too_large_to_tell_logits_apart():
    """fp64 rounds every candidate of a beam to the beam's score: within the beam the logits'
    order holds, equal beams go by number, and every place is filled."""
    dsa = lib()
    x = rand(2, 3, 5000, seed=3)
    got = run(dsa, x, [[-1e30, -1e30, -2e30], [-2e30, -1e30, -1e30]], None, 7, -1)
    for b, w in ((0, 0), (1, 1)):
        best = x[b, w].float().topk(7).indices.tolist()
        assert [(p, t) for p, t, _, _ in got[b]] == [(3 * b + w, t) for t in best]
        assert all(s == float(torch.tensor(-1e30)) for _, _, s, _ in got[b])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fill", [-1e4, -1e6, -1e9, -3e9, -1e10, -1e20, -1e30, -1e37, -3e38, 5e9, 1e30])
def test_finite_logits_of_any_size(fill, dtype):
    """Masks of a finite fill: a row that holds nothing else is uniform, one that holds other logits
    (if the fill is low) is as if they alone were there."""
    dsa = lib()
    V = 9000
    x = rand(2, 3, V, seed=7)
    x[0, 1] = fill
    x[0, 2, :8500] = fill                    # whole chunks, and part of one
    x[1, 0, ::3] = fill                      # some of each thread's
    x[1, 1, 100:] = fill
    x[1, 2, torch.arange(V) // 64 % 2 == 0] = fill  # all of some threads', none of others'
    check(dsa, x, [[-9.0, 0.0, -9.5], [-1.0, -2.0, -3.0]], None, 32, -1, dtype=dtype)
    check(dsa, x[:1, 1:2].contiguous(), [[-1.5]], None, 8, -1, dtype=dtype)


@pytest.mark.parametrize("size", [1e5, 3e6, 1e9, 2e9, 1e10, 1e20])
@pytest.mark.parametrize("sign", [-1, 1])
def test_large_logits_close_together(size, sign):
    # neighbours among the numbers of that size: whole steps of their last place apart
    dsa = lib()
    top = torch.tensor(sign * size, dtype=torch.float32)
    step = float((torch.nextafter(top, torch.tensor(math.inf)) - top).double())
    g = torch.Generator().manual_seed(3)
    x = float(top) - step * torch.randint(0, 400, (1, 2, 5000), generator=g).double() * max(1.0, round(0.01 / step))
    check(dsa, x, [[-3.0, -3.5]], None, 32, -1)


def test_scores_a_few_billionths_apart():
    """n equal logits: every term and sum is exact, a candidate's score is score - ln n.  Pairs of beams
    whose candidates differ by 1e-10 to 4e-9 are told apart (a logarithm is off by 2e-11 at most; an fp32
    one would be off by up to 3e-8)."""
    dsa = lib()
    rng = random.Random(1)
    cases = []
    while len(cases) < 200:
        a, b = rng.randrange(1, 4000), rng.randrange(1, 4000)
        sb = torch.tensor(rng.uniform(-2.0, -1.0)).item()
        sa = torch.tensor(sb + math.log(a) - math.log(b)).item()   # rounded to fp32
        if 1e-10 < abs((sa - sb) - (math.log(a) - math.log(b))) < 4e-9:
            cases.append((a, b, sa, sb))
    x = torch.full((len(cases), 2, 4000), -INF, dtype=torch.float64)
    for i, (a, b, _, _) in enumerate(cases):
        x[i, 0, :a] = x[i, 1, :b] = 0.0
    got = run(dsa, x, [[sa, sb] for _, _, sa, sb in cases], None, 1, -1)
    want = [int((sa - sb) < math.log(a) - math.log(b)) for a, b, sa, sb in cases]
    assert 50 < sum(want) < 150
    assert [g[0][0] - 2 * i for i, g in enumerate(got)] == want
