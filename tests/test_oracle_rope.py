"""Rotary positions' definition by hand, and the library's host-side frequencies against it."""
import math

import pytest
import torch

import oracle.rope as R


def test_hand_worked():
    # one pair, a quarter turn per position: (1, 2) -> (-2, 1) -> (-1, -2)
    quarter = [R.PI / 2]
    x = torch.tensor([[[9.0, 1.0, 2.0]], [[9.0, 1.0, 2.0]]], dtype=torch.float64)
    got = R.rope(x, [1, 2], quarter, 1, "half")
    assert torch.allclose(got, torch.tensor([[[9.0, -2, 1]], [[9, -1, -2]]], dtype=torch.float64), atol=1e-15)
    # two pairs, half layout (0, 2) and (1, 3) against neighbours
    y = torch.tensor([[[1.0, 2, 3, 4]]], dtype=torch.float64)
    f = [R.PI / 2, R.PI]
    assert torch.allclose(R.rope(y, [1], f, 0, "half"), torch.tensor([[[-3.0, -2, 1, -4]]], dtype=torch.float64))
    assert torch.allclose(R.rope(y, [1], f, 0, "interleaved"), torch.tensor([[[-2.0, 1, -3, -4]]], dtype=torch.float64))


def test_a_rotation_keeps_lengths_and_differences_of_positions():
    g = torch.Generator().manual_seed(1)
    f = R.frequencies(16, 10000.0)
    q, k = torch.randn(1, 1, 16, generator=g, dtype=torch.float64), torch.randn(1, 1, 16, generator=g, dtype=torch.float64)
    for layout in ("half", "interleaved"):
        dots = [float((R.rope(q, [a], f, 0, layout) * R.rope(k, [b], f, 0, layout)).sum())
                for a, b in ((5, 2), (1000005, 1000002), (0, -3))]
        assert max(dots) - min(dots) < 1e-12
        back = R.rope(R.rope(q, [77], f, 0, layout, 3.0), [77], f, 0, layout, 3.0, transposed=True)
        assert torch.allclose(back, 9 * q)


def test_scaling():
    plain = [float(x) for x in R.frequencies(64, 10000.0)]
    assert plain[0] == 1 and abs(plain[16] - 0.01) < 1e-15
    assert [float(x) * 4 for x in R.frequencies(64, 10000.0, "linear", 4.0)] == pytest.approx(plain, rel=1e-14)
    ntk = [float(x) for x in R.frequencies(64, 10000.0, "ntk", 4.0)]
    assert ntk[0] == 1 and ntk[-1] == pytest.approx(plain[-1] / 4, rel=1e-13)   # the last pair is stretched by the factor
    yarn = [float(x) for x in R.frequencies(64, 10000.0, "yarn", 40.0, 4096)]
    ratio = [a / b for a, b in zip(plain, yarn)]
    turns = [4096 * p / (2 * math.pi) for p in plain]
    assert all(r == pytest.approx(1, rel=1e-14) for r, t in zip(ratio, turns) if t > 40)
    assert all(r == pytest.approx(40, rel=1e-14) for r, t in zip(ratio, turns) if t < 0.8)
    assert all(a <= b * (1 + 1e-14) for a, b in zip(ratio, ratio[1:]))


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
    dict(scaling="yarn", factor=40.0, original=4096), dict(scaling="yarn", factor=1.0, original=131072),
    dict(scaling="yarn", factor=16.0, original=20), dict(scaling="yarn", factor=2.0, original=1 << 30, beta_fast=2.0)])
@pytest.mark.parametrize("rot_dim", [2, 26, 64, 256])
def test_the_librarys_steps(rot_dim, kw):
    """Steps are frequencies in 2^-64 turns; pow, the product and the quotients are each off by an ulp or two of 2^-53."""
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_long_gb300 as dsa
    r = dsa.make_rope(rot_dim=rot_dim, parts=[dsa.rope_part(heads=1, dim=rot_dim)], **kw)
    for i, f in enumerate(R.frequencies(rot_dim, **kw)):
        want = f / (2 * R.PI) * 2 ** 64
        assert abs(r.step[i] - want) <= want * 16 / 2 ** 53 + 1
