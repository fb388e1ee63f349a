"""Sampling's definition by hand."""
import math

from oracle.sample import kept_tokens, sample

INF, ln = math.inf, math.log


def test_hand_worked():
    x = [ln(4), ln(1), ln(2), ln(1)]                       # 1/2, 1/8, 1/4, 1/8
    draw = lambda u, **kw: sample(x, u, **kw)[0]
    assert [draw(u) for u in (0.0, 0.49, 0.51, 0.62, 0.63, 0.87, 0.88, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert abs(sample(x, 0.7)[1] - 0.25) < 1e-15
    # two largest; of equal ones the lower index
    assert [draw(u, top_k=2) for u in (0.66, 0.67)] == [0, 2]
    assert [draw(u, top_k=3) for u in (0.57, 0.58, 0.71, 0.72)] == [0, 1, 1, 2]
    # 1/2 does not reach 0.6, 3/4 does; of the two largest (2/3, 1/3) the first does
    assert [draw(u, top_p=0.6) for u in (0.66, 0.67)] == [0, 2]
    assert kept_tokens(x, 1.0, top_k=2, top_p=0.6)[0].tolist() == [0]
    assert kept_tokens(x, 1.0, top_p=1e-9)[0].tolist() == [0]
    # 1/4 of the largest is 1/8
    assert kept_tokens(x, 1.0, min_p=0.3)[0].tolist() == [0, 2] and kept_tokens(x, 1.0, min_p=0.2)[0].tolist() == [0, 1, 2, 3]
    # half the temperature squares the weights: 16, 1, 4, 1
    assert [draw(u, temperature=0.5) for u in (0.72, 0.73, 0.77, 0.78)] == [0, 1, 1, 2]


def test_greedy_and_unusable():
    assert sample([1.0, 3.0, 3.0], 0.9, temperature=0.0)[:2] == (1, 1.0)
    assert sample([-INF, math.nan, INF], 0.5)[:2] == (-1, 0.0)
    assert sample([INF, 0.0, math.nan, 0.0], 0.6)[0] == 3
    low = -3.4e38
    assert sample([low, low], 0.7)[:2] == (1, 0.5)
