"""Rotary positions: the definition, with frequencies and angles to 50 digits."""
from __future__ import annotations

import math
from decimal import Decimal, getcontext

import torch

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0):
    """Angle per position of each pair, as Decimals."""
    b, f, r = Decimal(base), Decimal(factor), rot_dim
    if scaling == "ntk" and r > 2:
        b = b * f ** (Decimal(r) / Decimal(r - 2))
    plain = [(-Decimal(2 * i) / r * b.ln()).exp() for i in range(r // 2)]
    if scaling == "linear":
        return [x / f for x in plain]
    if scaling != "yarn":
        return plain
    pair = lambda turns: r * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), r - 1)
    out = []
    for i, x in enumerate(plain):
        # 0: keeps its frequency, 1: stretched
        g = Decimal(0) if i <= low else Decimal(1) if i >= high else Decimal(i - low) / Decimal(high - low)
        out.append(x * (1 - g) + x / f * g)
    return out


def cos_sin(pos, freq):
    """fp64 tensors [len(pos), len(freq)]; the angle is reduced to one turn in decimal arithmetic."""
    turn = [[(Decimal(p) * f / (2 * PI)) % 1 for f in freq] for p in pos]
    angle = torch.tensor([[float(2 * PI * t) for t in row] for row in turn], dtype=torch.float64)
    return angle.cos(), angle.sin()


def rope(x, pos, freq, offset, layout, mscale=1.0, transposed=False):
    """x [n, H, D] -> fp64 [n, H, D], columns offset .. offset + 2 len(freq) rotated."""
    c, s = (mscale * t[:, None, :].to(x.device) for t in cos_sin(pos, freq))
    if transposed:
        s = -s
    out, h = x.double().clone(), len(freq)
    if layout == "half":
        i, j = slice(offset, offset + h), slice(offset + h, offset + 2 * h)
    else:
        i, j = slice(offset, offset + 2 * h, 2), slice(offset + 1, offset + 2 * h, 2)
    a, b = x[..., i].double(), x[..., j].double()
    out[..., i], out[..., j] = a * c - b * s, a * s + b * c
    return out
