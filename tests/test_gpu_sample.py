"""Sampling on the GPU against the fp64 definition.

Tokens must be equal.  A weight is off by 2^-29 of itself and one unit of 2^-44 of the
largest, so a part of the mass is off by less than 2^-28 + vocab 2^-44 times the largest
token's part of the mass; the inputs keep every draw and every border of top-p further than
that from a sum of weights (checked), or make all of them whole numbers of units.  A probability is off by 2^-27 and its rounding, 2^-24, relative.
"""
import math
import random
import threading

import pytest
import torch

from gpu_util import DEV, lib
from oracle.sample import kept_tokens, sample

pytestmark = pytest.mark.gpu
INF = math.inf
F32, BF16 = torch.float32, torch.bfloat16


def dev(x, dtype=F32):
    return None if x is None else torch.tensor(x, dtype=dtype, device=DEV)


def run(dsa, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, index=None, ld=None, dtype=F32, offset=0,
        stream=None):
    """logits [rows, V] (any float tensor) -> tokens, probabilities."""
    n, V = logits.shape
    ld = ld or V
    store = torch.full((n * ld + offset,), INF, dtype=dtype, device=DEV)    # what lies between the rows is not read
    x = store[offset:].view(n, ld)
    x[:, :V] = logits.to(dtype)
    settings = [temperature, top_k, top_p, min_p]
    m = next((len(t) for t in settings if t is not None), n)
    s = dsa.make_sampler(rows=n, vocab=V, ld=ld, dtype="bf16" if dtype == BF16 else "fp32", requests=m)
    token = torch.full((n,), 77, dtype=torch.int32, device=DEV)
    prob = torch.full((n,), math.nan, device=DEV)
    dsa.sample(s, x, dev(u), dev(temperature), dev(top_k, torch.int32), dev(top_p), dev(min_p), dev(index, torch.int32),
               token, prob, stream=stream)
    torch.cuda.synchronize()
    return token.tolist(), prob.tolist()


def check(dsa, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, index=None, dtype=F32, exact=False, **kw):
    tokens, probs = run(dsa, logits, u, temperature, top_k, top_p, min_p, index, dtype=dtype, **kw)
    assert dsa.get_status() == 0
    x = logits.to(dtype).double().numpy()
    f32 = lambda t, i, default: default if t is None else float(torch.tensor(t[i], dtype=F32))
    for r in range(x.shape[0]):
        q = r if index is None else index[r]
        cuts = f32(temperature, q, 1.0), 0 if top_k is None else top_k[q], f32(top_p, q, 1.0), f32(min_p, q, 0.0)
        want, p, margin = sample(x[r], f32(u, r, 0), *cuts)
        largest = 1 / max(1.0, float(kept_tokens(x[r], *cuts)[1].sum()))
        assert exact or margin > 2.0 ** -28 + x.shape[1] * 2.0 ** -44 * largest
        assert tokens[r] == want, (r, tokens[r], want, margin)
        assert abs(probs[r] - p) <= p * 2.0 ** -23


def rand(*shape, seed=0, scale=2.5):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * scale


def uniform(n, seed=0):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed)).tolist()


SETTINGS = [dict(), dict(temperature=[0.0]), dict(temperature=[0.7]), dict(temperature=[3.0], top_k=[1]),
            dict(top_k=[7]), dict(top_k=[50], top_p=[0.9]), dict(top_k=[3000]), dict(top_p=[0.95]), dict(top_p=[0.3]),
            dict(temperature=[1.3], min_p=[0.05]), dict(temperature=[0.9], top_k=[40], top_p=[0.8], min_p=[0.02]),
            dict(top_p=[0.999], min_p=[1e-4])]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,ld,offset", [(1, None, 0), (2, None, 0), (5, 7, 1), (100, None, 0), (1000, 1008, 0), (4099, None, 3),
                                         (8192, None, 0), (32001, 32008, 0), (70001, None, 0), (131071, 131072, 0)])
def test_settings_and_sizes(V, ld, offset, dtype):
    dsa = lib()
    rows = 4 if V < 50000 else 2
    x = rand(rows, V, seed=V)
    for i, s in enumerate(SETTINGS):
        kw = {k: v * rows for k, v in s.items()}
        check(dsa, x, uniform(rows, seed=1000 * i + V), ld=ld, dtype=dtype, offset=offset, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("spread", [0.01, 1.0, 8.0])
def test_rows_of_many_requests(spread, dtype):
    dsa = lib()
    n, m, V = 120, 7, 5003
    rng = random.Random(int(100 * spread))
    check(dsa, rand(n, V, seed=3, scale=spread), uniform(n, seed=9), index=[rng.randrange(m) for _ in range(n)], dtype=dtype,
          temperature=[0.0, 0.5, 0.8, 1.0, 1.2, 0.3, 2.0], top_k=[0, 0, 1, 30, 500, 5003, 6000],
          top_p=[1.0, 0.9, 1.0, 0.5, 0.99, 0.7, 0.01], min_p=[0.0, 0.1, 0.0, 0.0, 0.001, 1.0, 0.0])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ties(dtype):
    """Equal logits: weights are whole, every border is exact; those kept are the lowest."""
    dsa = lib()
    V = 1 << 15
    x = torch.zeros(6, V, dtype=torch.float64)
    u = [0.0, 0.25, 0.5, 1 - 2.0 ** -15, 1 - 2.0 ** -24, 2.0 ** -15]
    check(dsa, x, u, dtype=dtype, exact=True)
    check(dsa, x, u, dtype=dtype, exact=True, top_k=[1, 3, 4, 1000, 20000, 32767])
    check(dsa, x, u, dtype=dtype, exact=True, top_p=[2.0 ** -15, 0.25, 0.5, 2.0 ** -10, 0.75, 1.0])
    check(dsa, x, u, dtype=dtype, exact=True, top_k=[4, 8, 16, 1024, 16384, 2], top_p=[0.5, 0.25, 0.75, 1.0, 0.5, 0.5])
    check(dsa, x, u, dtype=dtype, exact=True, min_p=[1.0] * 6, temperature=[0.0, 1.0, 2.0, 3.0, 0.1, 1e-3])
    check(dsa, (rand(8, 30000, seed=2).round() * 0.5), uniform(8, seed=5), dtype=dtype, top_k=[1, 2, 20, 300, 4000, 0, 0, 9],
          top_p=[1.0, 1.0, 0.9, 0.8, 0.7, 0.6, 0.5, 0.4])          # many equal logits
    signed = torch.zeros(1, 300, dtype=torch.float64)
    signed[:, ::2] = -0.0                                          # -0 and +0 are one value
    check(dsa, signed, [0.55], dtype=dtype, top_k=[256], exact=True)
    check(dsa, torch.cat([signed, torch.tensor([[-1.0, -2.0]])], 1), [0.55], dtype=dtype, top_p=[0.5])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_and_unusable_logits(dtype):
    dsa = lib()
    x = rand(6, 9000, seed=4)
    x[0, 10:] = -INF                         # fewer logits than top_k
    x[1] = -INF                              # none
    x[2, 5], x[2, 6], x[2, 8999] = INF, math.nan, -INF
    x[3] = torch.finfo(dtype).min            # the type's lowest value is a logit like any other
    x[4, ::2] = math.nan
    x[5, :8500] = INF
    u = uniform(6, seed=2)
    for kw in (dict(), dict(top_k=[50] * 6), dict(top_p=[0.9] * 6), dict(min_p=[0.1] * 6), dict(temperature=[0.0] * 6)):
        check(dsa, x, u, dtype=dtype, **kw)
    assert run(dsa, x[1:2], [0.5], dtype=dtype) == ([-1], [0.0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fill", [-1e4, -1e9, -1e30, -3e38, 5e9, 1e30])
def test_finite_logits_of_any_size(fill, dtype):
    dsa = lib()
    V = 9000
    x = rand(4, V, seed=7)
    x[0] = fill
    x[1, :8500] = fill
    x[2, ::3] = fill
    x[3, 100:] = fill
    u = [0.50317, 0.30023, 0.70041, 0.12343]
    for kw in (dict(), dict(top_k=[40] * 4, top_p=[0.91] * 4), dict(top_p=[0.81234] * 4), dict(temperature=[1e7, 0.5, 2.0, 1.0])):
        check(dsa, x, u, dtype=dtype, **kw)


@pytest.mark.parametrize("T", [1e-30, 1e-6, 0.01, 100.0, 1e6, 1e30])
def test_extreme_temperatures(T):
    dsa = lib()
    x = rand(3, 5000, seed=11, scale=4.0)
    check(dsa, x, [0.20031, 0.50071, 0.90013], temperature=[T] * 3)
    check(dsa, x, [0.20031, 0.50071, 0.90013], temperature=[T] * 3, top_p=[0.9131] * 3, top_k=[101] * 3)


def test_a_large_spread_of_small_differences():
    """Logits of some 1e5 apart by a few units of their last place (2^-7): the difference comes first."""
    dsa = lib()
    g = torch.Generator().manual_seed(3)
    x = 1e5 - 2.0 ** -7 * torch.randint(0, 400, (3, 5000), generator=g).double()
    check(dsa, x, [0.1, 0.6, 0.95])
    check(dsa, x, [0.1, 0.6, 0.95], top_p=[0.5] * 3, temperature=[0.7] * 3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [3, 600])
def test_probabilities_of_light_tokens(n, dtype):
    """u = 0 draws token 0, 2^-10 to 2^-30 of the largest weight (units of 2^-58 of that: 2^-28 of it at most)."""
    dsa = lib()
    g = torch.Generator().manual_seed(n)
    T = (0.02 * 100 ** torch.rand(n, generator=g)).tolist()
    x = torch.rand(n, 9, generator=g, dtype=torch.float64) * -4.0
    t = torch.tensor(T, dtype=torch.float64)[:, None]
    top = torch.rand(n, 1, generator=g, dtype=torch.float64) * 26.0 - 13.0
    x = top + x * t
    x[:, 4:5] = top
    x[:, 0:1] = top - (10 + 19 * torch.rand(n, 1, generator=g, dtype=torch.float64)) * math.log(2) * t
    for cuts in (dict(), dict(top_k=[9] * n), dict(min_p=[2.0 ** -40] * n)):
        check(dsa, x, [0.0] * n, temperature=T, dtype=dtype, exact=True, **cuts)


def test_every_cdf_step_of_a_small_row():
    """u in the middle of each token's part of the mass, and a hair below its end."""
    dsa = lib()
    V = 257
    x = rand(1, V, seed=21)
    w = torch.exp(x[0].float().double() - x.max())
    c = torch.cumsum(w, 0) / w.sum()
    mid = (c - 0.5 * w / w.sum()).float().tolist()
    assert run(dsa, x.expand(V, V), mid)[0] == list(range(V))
    end = (c - 2.0 ** -22).float().tolist()
    assert run(dsa, x.expand(V, V), end)[0] == list(range(V))


def test_frequencies_follow_the_distribution():
    """4,096 evenly spaced draws: a token's count is its part of the mass, to one at either end."""
    dsa = lib()
    n, V = 4096, 40
    x = rand(1, V, seed=22, scale=1.0)
    u = [(i + 0.5) / n for i in range(n)]
    tokens, _ = run(dsa, x.expand(n, V), u, temperature=[0.8] * n, top_p=[0.9] * n)
    kept, w, _ = kept_tokens(x[0].float().double().numpy(), float(torch.tensor(0.8)), 0, float(torch.tensor(0.9)))
    count = torch.bincount(torch.tensor(tokens), minlength=V)
    assert int(count.sum()) == int(count[kept.tolist()].sum()) == n
    for t, part in zip(kept.tolist(), w / w.sum()):
        assert abs(int(count[t]) - n * part) <= 1 + n * 2.0 ** -23


MANY = 170                                       # rows enough for a CTA each


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,ld,offset", [(1, None, 0), (3, 5, 1), (100, None, 0), (257, 260, 3), (2049, None, 0), (4096, None, 0),
                                         (8193, 8200, 0), (12007, None, 2), (40001, None, 0)])
def test_many_rows_of_every_kind(V, ld, offset, dtype):
    """Rows with a small top_k or min_p, and among them all others."""
    dsa = lib()
    rng = random.Random(V)
    pick = lambda *v: [rng.choice(v) for _ in range(MANY)]
    u = uniform(MANY, seed=V + 1)
    kw = dict(temperature=pick(0.0, 0.7, 1.0, 1.3), top_k=pick(0, 1, 2, 7, 40, 100, 192, 193, 400, V),
              top_p=pick(1.0, 1.0, 0.9, 0.51, 0.99), min_p=pick(0.0, 0.0, 0.05, 0.3, 1.0))
    check(dsa, rand(MANY, V, seed=V), u, ld=ld, dtype=dtype, offset=offset, **kw)
    check(dsa, rand(MANY, V, seed=V + 5, scale=0.3), u, ld=ld, dtype=dtype, offset=offset, top_k=[min(50, V)] * MANY)
    check(dsa, rand(MANY, V, seed=V + 6), u, ld=ld, dtype=dtype, offset=offset, min_p=[0.02] * MANY)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_with_ties_and_masks(dtype):
    """More candidates than can be listed; logits in ascending and descending order; masked rows."""
    dsa = lib()
    V = 1 << 15
    u = uniform(MANY, seed=3)
    ks = [1 + (7 * i) % 192 for i in range(MANY)]
    flat = torch.zeros(MANY, V, dtype=torch.float64)
    exact_u = [float(i % 64) / 64 for i in range(MANY)]
    check(dsa, flat, exact_u, dtype=dtype, top_k=[1 << (i % 8) for i in range(MANY)], exact=True)
    check(dsa, flat, exact_u, dtype=dtype, min_p=[1.0] * MANY, exact=True)
    check(dsa, flat, [0.5] * MANY, dtype=dtype, top_k=[64] * MANY, temperature=[0.0] * MANY, exact=True)
    ramp = (torch.arange(V, dtype=torch.float64) / 512).expand(MANY, V)
    for x in (ramp, -ramp, (rand(MANY, V, seed=8).round() * 0.5)):
        check(dsa, x, u, dtype=dtype, top_k=ks, top_p=[0.97] * MANY)
    x = rand(MANY, 9000, seed=4)
    for r in range(MANY):
        kind = r % 8
        if kind == 0:
            x[r, 5:] = -INF                      # fewer logits than top_k
        elif kind == 1:
            x[r] = -INF                          # none
        elif kind == 2:
            x[r, ::2] = math.nan
        elif kind == 3:
            x[r, 1000:8500] = INF
        elif kind == 4:
            x[r] = torch.finfo(dtype).min
        elif kind == 5:
            x[r, :8900] = -1e9
    check(dsa, x, u, dtype=dtype, top_k=ks)
    check(dsa, x, u, dtype=dtype, min_p=[0.1] * MANY)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("begin", ["ascending", "lowest", "-1e4", "-3", "-inf"])
def test_many_rows_whose_bound_rises(begin, dtype):
    """The first logits of a row say little about the k-th largest: the bound rises by up to all of the type's range."""
    dsa = lib()
    n, V = 160, 30000
    x = rand(n, V, seed=31)
    if begin == "ascending":
        x = x.sort().values
    else:
        x[:, :20000] = float(torch.finfo(dtype).min) if begin == "lowest" else float(begin)
        x[:, :20000:3000] -= 0.5
    index = [r % 4 for r in range(n)]
    check(dsa, x, uniform(n, seed=32), index=index, dtype=dtype, top_k=[2, 40, 190, 1], top_p=[0.9, 0.95, 1.0, 1.0],
          temperature=[1.0, 0.8, 1.3, 1.0])
    check(dsa, -x.abs() if begin == "ascending" else x, uniform(n, seed=33), index=index, dtype=dtype,
          min_p=[0.05, 0.3, 0.01, 1.0])


def test_many_rows_as_a_graph():
    dsa = lib()
    n, V = 400, 9001
    s = dsa.make_sampler(rows=n, vocab=V, dtype="bf16", requests=3)
    x, u = torch.zeros(n, V, dtype=BF16, device=DEV), torch.zeros(n, device=DEV)
    k, p, i = dev([20, 0, 500], torch.int32), dev([0.9, 0.8, 1.0]), torch.zeros(n, dtype=torch.int32, device=DEV)
    token, prob = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, device=DEV)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        dsa.sample(s, x, u, None, k, p, None, i, token, prob)
    f = lambda v: float(torch.tensor(v, dtype=F32))
    for seed in range(2):
        y, r, q = rand(n, V, seed=seed).to(BF16), uniform(n, seed), [(j + seed) % 3 for j in range(n)]
        for t, v in ((x, y), (u, torch.tensor(r)), (i, torch.tensor(q))):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        want = [sample(y[j].double().numpy(), f(r[j]), 1.0, [20, 0, 500][q[j]], f([0.9, 0.8, 1.0][q[j]])) for j in range(n)]
        assert token.tolist() == [w[0] for w in want]
        assert all(abs(a - w[1]) <= w[1] * 2.0 ** -23 for a, w in zip(prob.tolist(), want))


@pytest.mark.parametrize("V,spread,T", [(131071, 1.0, 1.0), (131071, 2.5, 0.7), (100003, 0.05, 1.0), (60000, 3.0, 100.0),
                                        (60000, 3.0, 1e6), (200000, 1.0, 1.0), (30011, 6.0, 1.0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_nuclei(V, spread, T, dtype):
    """Cuts among many logits: many different ones, few different ones (bf16 values in either type), and more
    near the cut than can be listed."""
    dsa = lib()
    x = rand(3, V, seed=V, scale=spread)
    x[1] = x[1].to(BF16).double()
    u = uniform(3, seed=V + 1)
    for kw in (dict(top_p=[0.9, 0.8, 0.99]), dict(top_p=[0.3, 0.6, 0.95], top_k=[V // 2, V // 3, 5000]),
               dict(top_k=[V // 2, 1025, V - 1]), dict(top_p=[0.9703] * 3, min_p=[0.01, 0.001, 0.0])):
        check(dsa, x, u, dtype=dtype, temperature=[T] * 3, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [900, 20011, 131071])
def test_cold_rows(V, dtype):
    """Logits / temperature in the thousands: few tokens weigh anything, or many equal ones do."""
    dsa = lib()
    x = rand(12, V, seed=V + 1, scale=4.0)
    x[6:9] += 1000.0
    x[9:] = (x[9:] * 0.25).round() * 4.0
    x[11] = 40.0
    T = [0.01, 0.003, 0.0005, 0.01, 0.02, 0.003, 1.0, 0.7, 0.05, 0.01, 0.001, 0.02]
    u = [0.5 + 2.0 ** -12] * 3 + uniform(8, seed=V + 5) + [0.75]
    for p in (0.91, 0.23):
        check(dsa, x[:11], u[:11], temperature=T[:11], top_p=[p] * 11, dtype=dtype)
    check(dsa, x[:11], u[:11], temperature=T[:11], top_k=[300] * 11, top_p=[0.95] * 11, dtype=dtype)
    check(dsa, x[:11], u[:11], temperature=T[:11], top_k=[V // 2] * 11, dtype=dtype)
    check(dsa, x[11:], u[11:], temperature=T[11:], top_p=[0.5], dtype=dtype, exact=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_wanted_than_there_are(dtype):
    """A large top_k over a row with few usable logits, in every form of the call."""
    dsa = lib()
    x = rand(3, 20000, seed=9)
    x[0, 1500:] = -INF
    x[1, ::3], x[1, 1::3] = math.nan, INF
    x[2, 7:] = -INF
    u = uniform(3, seed=4)
    for kw in (dict(top_k=[1501, 19999, 8]), dict(top_k=[1500, 6666, 7]), dict(top_k=[5000, 6000, 2000], top_p=[0.9] * 3),
               dict(top_p=[0.95] * 3), dict(top_p=[0.95] * 3, min_p=[1e-3] * 3), dict(top_k=[1499, 6665, 6])):
        check(dsa, x, u, dtype=dtype, **kw)
    many = x.repeat(60, 1)
    check(dsa, many, uniform(180, seed=5), dtype=dtype, top_k=[150, 190, 8] * 60)


def test_two_calls_at_once():
    """Nothing is shared between calls: two streams, many rows each."""
    dsa = lib()
    n, V = 300, 5001
    s = dsa.make_sampler(rows=n, vocab=V, dtype="fp32")
    xs = [rand(n, V, seed=40 + i).float().to(DEV) for i in range(2)]
    us, k, p = [dev(uniform(n, seed=50 + i)) for i in range(2)], dev([30, 0, 300] * 100, torch.int32), dev([0.9, 0.95, 1.0] * 100)
    want = []
    for x, u in zip(xs, us):
        t = torch.zeros(n, dtype=torch.int32, device=DEV)
        dsa.sample(s, x, u, None, k, p, None, None, t)
        want.append(t)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [torch.zeros(n, dtype=torch.int32, device=DEV) for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                dsa.sample(s, xs[i], us[i], None, k, p, None, None, got[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and dsa.get_status() == 0


def test_settings_out_of_range():
    dsa = lib()
    x = rand(8, 100, seed=1)
    u = [0.5] * 8
    bad = [-1, 0.0]
    good, _ = run(dsa, x, u)
    for kw in (dict(temperature=[1, -0.5, math.nan, INF, 1, 1, 1, 1]), dict(top_k=[0, -1, -5, -2 ** 31, 0, 0, 0, 0]),
               dict(top_p=[1, 0, 1.5, math.nan, 1, 1, 1, 1]), dict(min_p=[0, -0.1, 1.1, math.nan, 0, 0, 0, 0])):
        t, p = run(dsa, x, u, **kw)
        assert dsa.get_status() == dsa.DSA_ERR_INDEX
        assert t == [good[0], -1, -1, -1] + good[4:] and p[1:4] == [0.0] * 3
    t, _ = run(dsa, x, [0.5, 1.0, -0.1, math.nan] + u[4:])
    assert dsa.get_status() == dsa.DSA_ERR_INDEX and t == [good[0], -1, -1, -1] + good[4:]
    t, _ = run(dsa, x, u, temperature=[1.0] * 3, index=[0, 3, -1, 2 ** 31 - 1, 0, 1, 2, 0])
    assert dsa.get_status() == dsa.DSA_ERR_INDEX and t == [good[0], -1, -1, -1] + good[4:]
    # a greedy row uses neither u nor the other settings
    t, p = run(dsa, x, [math.nan] * 8, temperature=[0.0] * 8, top_p=[-1.0] * 8, top_k=[-1] * 8, min_p=[2.0] * 8)
    assert dsa.get_status() == 0 and t == x.float().argmax(1).tolist() and p == [1.0] * 8


def test_a_row_gives_the_same_bits_wherever_it_lies():
    dsa = lib()
    x = rand(1, 7003, seed=5)
    for dtype in (F32, BF16):
        seen = set()
        for ld, offset in ((None, 0), (7008, 0), (7004, 1), (7003, 5), (9001, 2)):
            t, p = run(dsa, x.expand(3, 7003), [0.37] * 3, temperature=[0.9] * 3, top_p=[0.93] * 3, ld=ld, offset=offset,
                       dtype=dtype)
            seen |= set(zip(t, p))
        assert len(seen) == 1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cuts", [dict(min_p=0.0045), dict(top_k=200, top_p=0.97), dict(top_p=0.8), dict()])
def test_a_row_gives_the_same_bits_in_any_batch(cuts, dtype):
    """One row is spread over eight CTAs, 200 take one each; what is kept lies all in the first CTA's part."""
    dsa = lib()
    n, V = 200, 40000
    x, u = rand(n, V, seed=77).sort(descending=True).values, uniform(n, seed=78)
    of = lambda m: {k: [v] * m for k, v in dict(cuts, temperature=0.93).items()}
    want = list(zip(*run(dsa, x, u, dtype=dtype, **of(n))))
    assert list(zip(*run(dsa, x[:40], u[:40], dtype=dtype, **of(40)))) == want[:40]
    for r in range(40):
        assert list(zip(*run(dsa, x[r:r + 1], u[r:r + 1], dtype=dtype, **of(1)))) == want[r:r + 1]
    assert dsa.get_status() == 0


def test_host_threads_with_different_sizes():
    dsa = lib()
    sizes = [(2, 200001), (3, 901), (1, 131071), (5, 30011)]
    calls = []
    for i, (n, V) in enumerate(sizes):
        calls.append((dsa.make_sampler(rows=n, vocab=V), rand(n, V, seed=90 + i).to(BF16).to(DEV), dev(uniform(n, seed=95 + i)),
                      dev([0.8] * n), torch.zeros(n, dtype=torch.int32, device=DEV)))
    sample = lambda c, token, stream: dsa.sample(c[0], c[1], c[2], None, None, c[3], None, None, token, stream=stream)
    for c in calls:
        sample(c, c[4], None)
    torch.cuda.synchronize()
    errors = []

    def work(c):
        try:
            stream, token = torch.cuda.Stream(), torch.zeros_like(c[4])
            for _ in range(200):
                sample(c, token, stream.cuda_stream)
            stream.synchronize()
            assert torch.equal(token, c[4])
        except Exception as e:
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and dsa.get_status() == 0


def test_graph_replay_on_new_logits_and_other_stream():
    dsa = lib()
    n, V = 5, 9001
    s = dsa.make_sampler(rows=n, vocab=V, dtype="fp32")
    x, u, k = torch.zeros(n, V, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    T, p, token = torch.ones(n, device=DEV), torch.ones(n, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        dsa.sample(s, x, u, T, k, p, None, None, token)
    for seed in range(3):
        y, r = rand(n, V, seed=seed), uniform(n, seed)
        ks, ps, ts = [0, 5, 100, 0, 2000], [0.9, 1.0, 0.8, 0.7, 0.95], [0.0, 1.0, 0.8, 1.2, 0.6]
        for t, v in ((x, y), (u, torch.tensor(r)), (k, torch.tensor(ks)), (p, torch.tensor(ps)), (T, torch.tensor(ts))):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        f = lambda v: float(torch.tensor(v, dtype=F32))
        want = [sample(y[i].float().double().numpy(), f(r[i]), f(ts[i]), ks[i], f(ps[i]))[0] for i in range(n)]
        assert token.tolist() == want
    assert run(dsa, y, r, ts, ks, ps, stream=side)[0] == want


def test_rows_past_four_gigabytes():
    dsa = lib()
    n, V, ld = 4, 1000, 800_000_000
    x = torch.zeros(n * ld, dtype=BF16, device=DEV).view(n, ld)
    y = rand(n, V, seed=1).to(BF16)
    x[:, :V] = y.to(DEV)
    token = torch.zeros(n, dtype=torch.int32, device=DEV)
    dsa.sample(dsa.make_sampler(rows=n, vocab=V, ld=ld), x, dev([0.3] * n), None, None, None, None, None, token)
    assert token.tolist() == [sample(y[i].double().numpy(), float(torch.tensor(0.3)))[0] for i in range(n)]


def test_largest_vocabulary_and_many_rows():
    dsa = lib()
    x = rand(1, 1 << 18, seed=31)
    for dtype in (F32, BF16):
        for i, kw in enumerate((dict(), dict(top_k=[60]), dict(top_p=[0.9]), dict(top_k=[100000], top_p=[0.95]))):
            check(dsa, x, [0.1 + 0.2 * i], dtype=dtype, **kw)
    n = 20000
    y = rand(1, 11, seed=32)
    u = torch.arange(n, dtype=F32) / n
    w = torch.exp(y[0].float().double() - y.float().max())
    want = torch.searchsorted(torch.cumsum(w, 0) / w.sum(), u.double(), right=True)
    assert run(dsa, y.expand(n, 11), u.tolist())[0] == want.tolist()


def test_refused_tensors():
    dsa = lib()
    n, V = 2, 8
    mk = lambda **kw: dsa.make_sampler(**dict(dict(rows=n, vocab=V, dtype="fp32"), **kw))
    x, u, token = torch.zeros(n, V, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    ok = dict(logits=x, u=u, temperature=None, top_k=None, top_p=None, min_p=None, index=None, token=token, prob=None)
    dsa.sample(mk(), **ok)
    for e, kw in ((TypeError, dict(logits=x.to(BF16))), (ValueError, dict(logits=x[:, :7])), (ValueError, dict(u=u[:1])),
                  (TypeError, dict(u=u.double())), (TypeError, dict(top_k=u)), (ValueError, dict(top_p=torch.ones(3, device=DEV))),
                  (ValueError, dict(min_p=u.cpu())), (TypeError, dict(index=u)), (TypeError, dict(token=token.long())),
                  (TypeError, dict(prob=token)), (TypeError, dict(token=None))):
        with pytest.raises(e):
            dsa.sample(mk(), **dict(ok, **kw))
    for s, kw in ((mk(requests=1), {}), (mk(), dict(prob=u)), (mk(), dict(index=token))):
        with pytest.raises(dsa.DSAError) as e:
            dsa.sample(s, **dict(ok, **kw))
        assert e.value.code == dsa.DSA_ERR_INVALID_ARG
    assert dsa.get_status() == 0


LIGHT = 2.0 ** -32                               # of the largest weight


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("light,front,k,min_p", [(2800, False, 5000, 0.0), (2800, True, 5000, 0.0), (500, False, 2000, 0.0),
                                                 (500, True, 1000, 0.0), (900, True, 1000, 0.0), (2000, False, 3000, 2.0 ** -34),
                                                 (5000, False, 19999, 0.0)])
def test_light_tokens_of_a_row_with_fewer_than_top_k(light, front, k, min_p, dtype):
    """One token, and others below 2^-32 of it, all kept: they count in the mass and are drawn.

    A weight is off by 2^-29 of itself and a unit of 2^-44 of the largest, so the mass before a token by a part of
    light * 2^-32 * 2^-29 + light * 2^-44 < 2^-30 at most: the drawn token's part of the mass must hold u to that.  A
    probability is off by as much of itself, a unit, and its rounding.
    """
    dsa = lib()
    n, V = 5, 20000
    g = torch.Generator().manual_seed(light + k)
    x = torch.full((n, V), -INF, dtype=torch.float64)
    for r in range(n):
        at = 1 + (torch.arange(light) if front else torch.randperm(V - 1, generator=g)[:light].sort().values)
        x[r, at] = -22.2 - 1.2 * torch.rand(light, generator=g, dtype=torch.float64) * (0.1 if light < 600 else 1.0)
        x[r, at[0]] = -22.2
        x[r, 0 if r < 3 else at[-1]] = 0.0       # in front of the light ones (u near 1 draws them) or behind (u = 0)
    u = [0.5, 1 - 2.0 ** -24, 1 - 2.0 ** -23, 0.0, 0.5]
    x = x.to(dtype).double()
    keep = dict(top_k=[k] * n, min_p=[min_p] * n)
    got = run(dsa, x, u, dtype=dtype, **keep)
    assert dsa.get_status() == 0
    drawn = 0
    for r in range(n):
        token, prob = got[0][r], got[1][r]
        kept, w, _ = kept_tokens(x[r].numpy(), 1.0, k, 1.0, min_p)
        part = dict(zip(kept.tolist(), (w / w.sum()).tolist()))
        before = math.fsum(part[t] for t in kept.tolist() if t < token)
        assert token in part and before - 2.0 ** -30 <= u[r] <= before + part[token] + 2.0 ** -30, (r, token)
        assert abs(prob - part[token]) <= part[token] * (2.0 ** -24 + 2.0 ** -30) + 2.0 ** -44, (r, prob, part[token])
        drawn += part[token] < LIGHT
    assert drawn >= 1
    # the same bits, whatever share of a row a CTA has and whatever kernel takes it
    for m in (20, 40):
        many = run(dsa, x.repeat(m, 1), u * m, dtype=dtype, top_k=[k] * n * m, min_p=[min_p] * n * m)
        assert many[0] == got[0] * m and many[1] == got[1] * m
    for r in range(n):
        one = run(dsa, x[r:r + 1], u[r:r + 1], dtype=dtype, top_k=[k], min_p=[min_p])
        assert one == (got[0][r:r + 1], got[1][r:r + 1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [2, 12, 200])
def test_a_number_added_to_all_logits_changes_nothing(n, dtype):
    """Logits on a grid that the type holds with every shift: the same tokens; in fp32 the same bits, as the
    difference to the largest comes first."""
    dsa = lib()
    V = 20011
    x = (rand(n, V, seed=61, scale=2.0) * 8).round().clamp(-56, 63) / 8   # -7 to 7.9 by eighths
    x += torch.where(torch.arange(V) % 1999 == 5, 7.0, 0.0)
    x.clamp_(max=12.0)
    u = uniform(n, seed=62)
    for kw in (dict(), dict(top_k=[40] * n), dict(top_k=[64] * n, top_p=[0.9013] * n), dict(min_p=[0.0137] * n),
               dict(top_p=[0.8021] * n), dict(top_k=[3000] * n), dict(temperature=[0.0] * n)):
        if n == 200:                             # (a row's result is compared with the definition's in the small batches)
            base = run(dsa, x, u, dtype=dtype, **kw)
        else:
            check(dsa, x, u, dtype=dtype, **kw)
            base = run(dsa, x, u, dtype=dtype, **kw)
        for shift in (-4.0, -8.0, -13.0, 8.0):
            tokens, probs = run(dsa, x + shift, u, dtype=dtype, **kw)
            assert tokens == base[0]
            if dtype == F32:
                assert probs == base[1]
            else:
                assert all(abs(a - b) <= b * 2.0 ** -23 for a, b in zip(probs, base[1]))
    assert dsa.get_status() == 0
