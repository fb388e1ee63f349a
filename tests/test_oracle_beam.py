"""Beam selection's definition by hand and against torch."""
import math

import torch

from oracle.beam import beam_select

INF = math.inf


def test_hand_worked():
    # two beams of probability (1/2, 1/4, 1/4) and (3/4, 1/4, 0) with scores ln 1/3 and ln 1/2:
    # candidates 1/6, 1/12, 1/12 and 3/8, 1/8
    ln = math.log
    got = beam_select([[[ln(2), 0.0, 0.0], [ln(3), 0.0, -INF]]], [[ln(1 / 3), ln(1 / 2)]], None, 6, 2)
    assert [(p, t) for p, t, _, _ in got[0]] == [(1, 0), (0, 0), (1, 1), (0, 1), (0, 2), (-1, -1)]
    for (_, _, s, _), want in zip(got[0], (3 / 8, 1 / 6, 1 / 8, 1 / 12, 1 / 12)):
        assert abs(s - ln(want)) < 1e-12
    assert [f for _, _, _, f in got[0]] == [False, False, False, False, True, False]


def test_finished_dead_and_unusable():
    x = [[1.0, 2.0], [5.0, 5.0], [INF, 3.0], [math.nan, -INF]]
    got = beam_select([x], [[-1.0, -3.0, -INF, 0.0]], [[0, 1, 0, 0]], 4, 0)
    # beam 1 is finished: token 0 at its score; beam 2 is dead, beam 3 has no logit
    assert [(p, t) for p, t, _, _ in got[0]] == [(0, 1), (0, 0), (1, 0), (-1, -1)]
    assert got[0][2][2] == -3.0 and got[0][2][3]
    got = beam_select([[[INF, 3.0, 3.0]]], [[0.0]], None, 3, -1)
    assert [t for _, t, _, _ in got[0]] == [1, 2, -1] and abs(got[0][0][2] + math.log(2)) < 1e-12


def test_against_log_softmax():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(2, 3, 50, generator=g, dtype=torch.float64)
    s = torch.randn(2, 3, generator=g, dtype=torch.float64)
    cand = (s[..., None] + torch.log_softmax(x, -1)).reshape(2, -1)
    best, at = cand.topk(7)
    got = beam_select(x.tolist(), s.tolist(), None, 7, -1)
    for b in range(2):
        assert [(p - 3 * b) * 50 + t for p, t, _, _ in got[b]] == at[b].tolist()
        assert torch.allclose(torch.tensor([r[2] for r in got[b]], dtype=torch.float64), best[b])
