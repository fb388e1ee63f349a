"""Beam selection in plain Python floats (fp64): the definition of dsa_beam_select."""
from __future__ import annotations

import math


def beam_select(logits, scores, finished, keep, eos):
    """logits: per request, per beam, a list of floats.  Returns per request a list of `keep`
    (parent row, token, score, finished), best first."""
    out = []
    for b, beams in enumerate(logits):
        cand = []
        for w, x in enumerate(beams):
            s = scores[b][w]
            if not s > -math.inf:
                continue
            if finished is not None and finished[b][w]:
                cand.append((-s, w * len(x) + eos, w, eos, s))
                continue
            ok = [v for v, t in enumerate(x) if -math.inf < t < math.inf]
            if not ok:
                continue
            top = max(x[v] for v in ok)
            # (x - top first: added to a large maximum the logarithm would be lost)
            ln = math.log(math.fsum(math.exp(x[v] - top) for v in ok))
            cand += [(-(s + ((x[v] - top) - ln)), w * len(x) + v, w, v, s + ((x[v] - top) - ln)) for v in ok]
        cand.sort()
        rows = [(b * len(beams) + w, v, s, bool((finished is not None and finished[b][w]) or v == eos))
                for _, _, w, v, s in cand[:keep]]
        out.append(rows + [(-1, -1, -math.inf, False)] * (keep - len(rows)))
    return out
