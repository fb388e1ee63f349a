"""Rotary positions on the GPU against the definition.

A sine or cosine is off by at most 4 half-steps of 2^-24: the angle's rounding to fp32
(pi 2^-25), to 2^-32 turns, and the function's own ulp (2^-24); with the steps' 53 bits an
angle is off by |pos| f 2^-51 more.  Times mscale, a product and a sum: four roundings of
2^-24.  So a result is off by (|a| + |b|) mscale (2^-21 + |pos| f 2^-51), and then rounded
to its type.
"""
import math
import random

import pytest
import torch

import oracle.rope as R
from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def rand(*shape, seed=0, dtype="fp32"):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(TYPE[dtype]).to(DEV)


def check(got, x, pos, freq, offset, layout, dtype, mscale=1.0, transposed=False):
    """got, x: [n, H, D]."""
    want = R.rope(x, pos, freq, offset, layout, mscale, transposed)
    h, r = len(freq), 2 * len(freq)
    rot = slice(offset, offset + r)
    y = x[..., rot].double().abs()
    if layout == "half":
        both = (y[..., :h] + y[..., h:]).repeat(1, 1, 2)
        f = torch.tensor([float(v) for v in freq] * 2, dtype=torch.float64, device=DEV)
    else:
        both = (y[..., 0::2] + y[..., 1::2]).repeat_interleave(2, -1)
        f = torch.tensor([float(v) for v in freq], dtype=torch.float64, device=DEV).repeat_interleave(2)
    far = torch.tensor(pos, dtype=torch.float64, device=DEV).abs()[:, None, None] * f
    tol = both * abs(mscale) * (2.0 ** -21 + far * 2.0 ** -51) + HALF_STEP[dtype] * want[..., rot].abs()
    assert bool(((got[..., rot].double() - want[..., rot]).abs() <= tol).all())
    for rest in (slice(0, offset), slice(offset + r, None)):
        assert torch.equal(got[..., rest], x[..., rest])


FAR = [0, 1, -1, 4096, 131071, 1 << 20, 16777217, (1 << 31) - 1, -(1 << 31)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,H,D,rot,offset,kw", [
    (1, 1, 2, 2, 0, {}), (9, 3, 7, 4, 3, {}), (5, 128, 576, 64, 512, dict(scaling="yarn", factor=40.0, original=4096)),
    (17, 1, 576, 64, 512, {}), (33, 64, 128, 64, 0, dict(mscale=1.2)), (2, 5, 80, 26, 0, dict(scaling="linear", factor=8.0)),
    (130, 2, 64, 64, 0, dict(scaling="ntk", factor=4.0)), (3, 2, 256, 256, 0, {}), (4, 3, 300, 8, 291, {}),
    (2, 2, 5000, 32, 8, {}), (700, 1, 16, 16, 0, {})])
def test_in_and_out_of_place_both_ways(n, H, D, rot, offset, kw, dtype, layout):
    dsa = lib()
    rng = random.Random(n * D)
    pos = [rng.choice(FAR) if i % 3 else rng.randrange(200000) for i in range(n)]
    m = kw.get("mscale", 1.0)
    freq = R.frequencies(rot, **{k: v for k, v in kw.items() if k != "mscale"})
    r = dsa.make_rope(rot_dim=rot, parts=[dsa.rope_part(heads=H, dim=D, offset=offset, layout=layout, dtype=dtype)], **kw)
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)
    x = rand(n, H, D, seed=D, dtype=dtype)
    for transposed in (False, True):
        out = torch.full_like(x, math.nan)
        dsa.rope_apply(r, p, (x,), (out,), transposed=transposed)
        check(out, x, pos, freq, offset, layout, dtype, m, transposed)
        y = x.clone()
        dsa.rope_apply(r, p, [y], transposed=transposed)
        assert torch.equal(y, out)
    assert dsa.get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_slices_orders_and_alignment(shift, dtype):
    """Columns out of wider rows, heads before tokens, rows that begin at any element; what lies between stays."""
    dsa = lib()
    n, H, rot = 11, 6, 32
    freq, pos = R.frequencies(rot), list(range(7, 7 + n))
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)
    for layout in ("half", "interleaved"):
        r = dsa.make_rope(rot_dim=rot, parts=[dsa.rope_part(heads=H, dim=rot, layout=layout, dtype=dtype)])
        x = rand(n, H, 96 + shift, seed=1, dtype=dtype)[..., 64 + shift:]
        store = torch.full((H, n, 160), 3.0, dtype=TYPE[dtype], device=DEV)
        out = store[..., 100 + shift:100 + shift + rot].transpose(0, 1)
        dsa.rope_apply(r, p, (x,), (out,))
        check(out, x, pos, freq, 0, layout, dtype)
        store[..., 100 + shift:100 + shift + rot] = 3.0
        assert bool((store == 3.0).all())
        # one row for all heads, [batch, sequence, heads, columns], and in place within a wider row
        one = rand(n, 1, rot, seed=2, dtype=dtype).expand(n, H, rot)
        out = torch.empty(1, n, H, rot, dtype=TYPE[dtype], device=DEV)
        dsa.rope_apply(r, p, (one,), (out,))
        check(out[0], one, pos, freq, 0, layout, dtype)
        wide = rand(n, H, 2 * rot + shift, seed=3, dtype=dtype)
        before = wide.clone()
        dsa.rope_apply(r, p, (wide[..., shift:shift + rot],))
        check(wide[..., shift:shift + rot], before[..., shift:shift + rot], pos, freq, 0, layout, dtype)
        assert torch.equal(wide[..., shift + rot:], before[..., shift + rot:])
        assert torch.equal(wide[..., :shift], before[..., :shift])


def latent_parts(dsa, shared="bf16"):
    return [dsa.rope_part(heads=128, dim=576, offset=512), dsa.rope_part(heads=1, dim=576, offset=512, dtype=shared),
            dsa.rope_part(heads=64, dim=128, layout="half"), dsa.rope_part(heads=1, dim=128, layout="half", dtype=shared)]


LATENT = [(128, 576, 512, "interleaved"), (1, 576, 512, "interleaved"), (64, 128, 0, "half"), (1, 128, 0, "half")]


def test_four_tensors_of_a_layer_as_a_graph_on_another_stream():
    dsa = lib()
    n, freq = 67, R.frequencies(64, scaling="yarn", factor=40.0, original=4096)
    r = dsa.make_rope(rot_dim=64, parts=latent_parts(dsa), scaling="yarn", factor=40.0, original=4096)
    x = [torch.zeros(n, H, D, dtype=torch.bfloat16, device=DEV) for H, D, _, _ in LATENT]
    x[1], x[3] = x[1][:, 0], x[3][:, 0]
    out = [torch.zeros_like(t) for t in x]
    p = torch.zeros(n, dtype=torch.int32, device=DEV)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        dsa.rope_apply(r, p, x, out)
    for seed in range(2):
        pos = [random.Random(seed).randrange(1 << 18) for _ in range(n)]
        p.copy_(torch.tensor(pos, dtype=torch.int32))
        for i, t in enumerate(x):
            t.copy_(rand(*t.shape, seed=10 * seed + i))
        g.replay()
        torch.cuda.synchronize()
        for t, o, (H, D, offset, layout) in zip(x, out, LATENT):
            check(o.view(n, H, D), t.view(n, H, D), pos, freq, offset, layout, "bf16")
    with torch.cuda.stream(side):
        again = [torch.zeros_like(t) for t in x]
        dsa.rope_apply(r, p, x, again)
    other = [torch.zeros_like(t) for t in x]
    dsa.rope_apply(r, p, x, other, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(out, again, other))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_the_gradient_is_the_transposed_call(layout):
    """Against the formula: <R x, y> = <x, R' y>; and against differences of sum(y R x), which is linear in x: its
    difference quotient is exact up to roundings.  All of some 4,000 products and sums of unit normals in fp32."""
    dsa = lib()
    n, H, D, rot, offset = 13, 4, 80, 32, 24
    r = dsa.make_rope(rot_dim=rot, parts=[dsa.rope_part(heads=H, dim=D, offset=offset, layout=layout, dtype="fp32")],
                      mscale=1.3)
    p = torch.arange(1000, 1000 + n, dtype=torch.int32, device=DEV)
    x, y = rand(n, H, D, seed=1), rand(n, H, D, seed=2)
    fx, gy = torch.empty_like(x), torch.empty_like(x)
    dsa.rope_apply(r, p, (x,), (fx,))
    dsa.rope_apply(r, p, (y,), (gy,), transposed=True)
    left, right = (fx.double() * y.double()), (x.double() * gy.double())
    scale = float(left.abs().sum() + right.abs().sum())
    assert abs(float(left.sum() - right.sum())) <= scale * 2.0 ** -20
    for seed in range(5):
        d = rand(n, H, D, seed=20 + seed)
        fd = torch.empty_like(x)
        dsa.rope_apply(r, p, ((x + d),), (fd,))
        quotient = float((y.double() * (fd.double() - fx.double())).sum())
        inner = gy.double() * d.double()
        assert abs(quotient - float(inner.sum())) <= (scale + float(inner.abs().sum())) * 2.0 ** -18


def test_parts_of_one_buffer_in_place():
    """Queries and keys as columns of one projection, rotated where they lie; its other columns stay."""
    dsa = lib()
    n, H, Hk, D = 37, 8, 2, 64
    for dtype in ("bf16", "fp32"):
        both = rand(n, (H + 2 * Hk) * D, seed=5, dtype=dtype)
        before = both.clone()
        q, k = both[:, :H * D].view(n, H, D), both[:, H * D:(H + Hk) * D].view(n, Hk, D)
        r = dsa.make_rope(rot_dim=D, parts=[dsa.rope_part(heads=h, dim=D, layout="half", dtype=dtype) for h in (H, Hk)])
        pos = list(range(100, 100 + n))
        dsa.rope_apply(r, torch.tensor(pos, dtype=torch.int32, device=DEV), (q, k))
        f = R.frequencies(D)
        check(q, before[:, :H * D].view(n, H, D), pos, f, 0, "half", dtype)
        check(k, before[:, H * D:(H + Hk) * D].view(n, Hk, D), pos, f, 0, "half", dtype)
        assert torch.equal(both[:, (H + Hk) * D:], before[:, (H + Hk) * D:])


def test_many_passes_and_short_tables():
    """Enough rows for sixteen passes of a CTA, with one head (a table of few tokens) and with many."""
    dsa = lib()
    for n, H, rot in ((70001, 1, 256), (3001, 96, 64), (20011, 3, 32)):
        r = dsa.make_rope(rot_dim=rot, parts=[dsa.rope_part(heads=H, dim=rot)])
        x = rand(n, H, rot, seed=n, dtype="bf16")
        pos = torch.arange(n, dtype=torch.int32, device=DEV) * 17
        out = torch.empty_like(x)
        dsa.rope_apply(r, pos, (x,), (out,))
        i = torch.cat([torch.arange(40), torch.randint(0, n, (60,), generator=torch.Generator().manual_seed(1)),
                       torch.arange(n - 40, n)])
        check(out[i.to(DEV)], x[i.to(DEV)], pos.cpu()[i].tolist(), R.frequencies(rot), 0, "interleaved", "bf16")


def test_rows_past_four_gigabytes():
    dsa = lib()
    n, D, rot = 3, 64, 64
    store = torch.zeros(2 * 1_500_000_000 + D, dtype=torch.bfloat16, device=DEV)
    x = store.as_strided((n, 1, D), (1_500_000_000, D, 1))
    y = rand(n, 1, D, seed=4, dtype="bf16")
    x.copy_(y)
    r = dsa.make_rope(rot_dim=rot, parts=[dsa.rope_part(heads=1, dim=D)])
    dsa.rope_apply(r, torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV), (x,))
    check(x, y, [5, 6, 7], R.frequencies(rot), 0, "interleaved", "bf16")


def test_infinities_and_nan_stay_in_their_pair():
    dsa = lib()
    x = rand(1, 1, 16, seed=1)
    x[0, 0, 2], x[0, 0, 5] = math.inf, math.nan
    r = dsa.make_rope(rot_dim=16, parts=[dsa.rope_part(heads=1, dim=16, dtype="fp32")])
    out = torch.empty_like(x)
    dsa.rope_apply(r, torch.tensor([3], dtype=torch.int32, device=DEV), (x,), (out,))
    assert bool(torch.isfinite(out[0, 0, [0, 1, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15]]).all())
    assert not bool(torch.isfinite(out[0, 0, [2, 3, 4, 5]]).any())


def test_refused_tensors():
    dsa = lib()
    r = dsa.make_rope(rot_dim=8, parts=[dsa.rope_part(heads=2, dim=16)])
    p = torch.zeros(3, dtype=torch.int32, device=DEV)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    good = bf(3, 2, 16)
    for e, pos, x, out in ((TypeError, p, (good.float(),), None), (TypeError, p.long(), (good,), None),
                           (ValueError, p, (bf(3, 2, 15),), None), (ValueError, p, (bf(3, 16),), None),
                           (ValueError, p, (bf(4, 2, 16),), None), (ValueError, p, (bf(2, 3, 2, 16)[:, 1:2],), None),
                           (ValueError, p, (good, good), None), (ValueError, p, (good,), ()),
                           (ValueError, p, (bf(3, 2, 32)[..., ::2],), None), (ValueError, p, (good.cpu(),), None),
                           (TypeError, p, ([[0.0]],), None), (ValueError, p, (bf(3, 3, 2, 16)[:1, :, :, :].expand(3, 3, 2, 16),), None)):
        with pytest.raises(e):
            dsa.rope_apply(r, pos, x, out)
    wide = bf(3, 2, 17)
    for x, out in ((wide[..., 1:], wide[..., :16]), (good, good.view(3, 2, 16).flip(0)[:1].expand(3, 2, 16))):
        with pytest.raises((dsa.DSAError, ValueError)):
            dsa.rope_apply(r, p, (x,), (out,))
    assert dsa.get_status() == 0
