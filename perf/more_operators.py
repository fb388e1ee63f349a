"""Measured cases of the operators before and behind the attention: rotary
positions of its inputs (and of their gradients), sampling of tokens from
logits, and acceptance of drafted tokens.

``run`` computes an operator in its plain form (elementary torch operations) or,
with ``own`` true, through the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
# latent attention with an indexer: 128 + 64 projected query columns per head, rows of 512 + 64, index heads of 128
LATENT = dict(H=128, Hk=1, rot=64, nope=128, lat=512, HI=64, d_I=128, base=10000.0, scaling="yarn", factor=40.0,
              original=4096)
# plain heads, rotated in front, key heads shared
HEADS = dict(nope=0, lat=0, HI=0, d_I=0, base=500000.0, scaling="none", factor=1.0, original=4096)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # rotary positions of a layer's inputs
        # one generated token: latency
        dict(name="rope-token", op="rope", n_tok=1, far=131072, dtype="bf16", back=False, **LATENT),
        # drafted trees of a serving batch, 16 sequences of 48 tokens
        dict(name="rope-draft", op="rope", n_tok=768, far=131072, dtype="bf16", back=False, **LATENT),
        # a training sequence or a prompt
        dict(name="rope-prompt", op="rope", n_tok=16384, far=0, dtype="bf16", back=False, **LATENT),
        # the gradients of one: rows of the shared keys in fp32, the others bf16
        dict(name="rope-grad", op="rope", n_tok=8192, far=0, dtype="bf16", back=True, **LATENT),
        # part of each head, odd sizes, the exact type
        dict(name="rope-part", op="rope", n_tok=333, far=1000003, dtype="fp32", back=False, H=8, Hk=2, rot=26, dim=80,
             **HEADS),
        # sampling
        # one request, small vocabulary of odd size: latency
        dict(name="sample-one", op="sample", rows=1, vocab=32001, ld=32001, dtype="fp32", mode="usual", requests=0,
             spread=2.5),
        # a serving batch, every request with settings of its own
        dict(name="sample-batch", op="sample", rows=64, vocab=131071, ld=131072, dtype="bf16", mode="mixed",
             requests=0, spread=2.5),
        # rollouts at a temperature, nothing cut off
        dict(name="sample-free", op="sample", rows=256, vocab=131071, ld=131072, dtype="bf16", mode="free", requests=0,
             spread=2.5),
        # the nucleus alone, over a flat distribution
        dict(name="sample-nucleus", op="sample", rows=48, vocab=64000, ld=64000, dtype="fp32", mode="nucleus",
             requests=0, spread=1.5),
        # a token at each drafted position of 16 trees, settings per request
        dict(name="sample-draft", op="sample", rows=768, vocab=64000, ld=64000, dtype="bf16", mode="usual",
             requests=16, spread=2.5),
        # acceptance of drafted tokens
        # one request, a chain of drafts: latency
        dict(name="accept-one", op="accept", n_seqs=1, lo=5, hi=5, tree=False, match=0.8, pick=1),
        # a serving batch with trees of several sizes
        dict(name="accept-batch", op="accept", n_seqs=256, lo=17, hi=64, tree=True, match=0.7, pick=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    largest = {}
    for c in listed():
        w = work(c)
        a, b = largest.get(c["op"], (0, 0))
        largest[c["op"]] = (max(a, w["bytes"]), max(b, w["flops"]))
    while True:
        op = rng.choice(["rope", "rope", "sample", "sample", "sample", "accept"])
        if op == "rope":
            c = dict(op=op, n_tok=_log(rng, 1, 16384), far=rng.choice([0, _log(rng, 4096, 1 << 21)]),
                     back=rng.random() < 0.4)
            if rng.random() < 0.6:
                c.update(dtype="bf16", **dict(LATENT, H=rng.choice([1, 8, 16, 24, 64, 128]), HI=rng.choice([0, 32, 64]),
                                              rot=rng.choice([32, 64, 64, 128])))
            else:
                dim = rng.choice([64, 80, 96, 128, 192, 256])
                Hk = rng.choice([1, 2, 4, 8])
                c.update(dtype=rng.choice(["bf16", "fp32"]), H=Hk * rng.randrange(1, 9), Hk=Hk, dim=dim,
                         rot=rng.choice([dim, dim // 2, 2 * rng.randrange(1, dim // 2 + 1)]), **HEADS)
            c.update(scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=rng.choice([2.0, 8.0, 40.0]))
        elif op == "sample":
            vocab, rows = _log(rng, 1000, 200000), _log(rng, 1, 768)
            c = dict(op=op, rows=rows, vocab=vocab, ld=vocab if rng.random() < 0.5 else (vocab + 63) // 64 * 64,
                     dtype=rng.choice(["fp32", "bf16"]),
                     mode=rng.choice(["usual", "mixed", "mixed", "free", "nucleus", "greedy"]),
                     requests=0 if rng.random() < 0.6 else rng.randrange(1, rows + 1), spread=rng.uniform(1.0, 5.0))
        else:
            hi = _log(rng, 1, 130)
            c = dict(op=op, n_seqs=_log(rng, 1, 512), lo=rng.randrange(0, hi + 1), hi=hi, tree=rng.random() < 0.6,
                     match=rng.uniform(0.2, 0.95), pick=rng.randrange(1 << 30))
            if sum(_counts(c)) == 0:
                continue
        w = work(c)
        if w["bytes"] <= largest[op][0] and w["flops"] <= largest[op][1]:
            return c


_SIZE = {"bf16": 2, "fp32": 4}
_TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _parts(c):
    """Of each tensor of a rotary case: name, heads, columns before the rotated ones (x, out), width, layout, type.
    Width 0: only the rotated columns are handed over, as slices of x and out."""
    t = c["dtype"]
    shared = "fp32" if c["back"] else t  # gradients of rows that all heads share are sums
    if not c["lat"]:
        return [("q", c["H"], 0, 0, c["dim"], "half", t), ("k", c["Hk"], 0, 0, c["dim"], "half", shared)]
    x, o = (c["lat"], c["nope"]) if c["back"] else (c["nope"], c["lat"])
    parts = [("q", c["H"], x, o, 0, "interleaved", t), ("kv", 1, c["lat"], c["lat"], 0, "interleaved", shared)]
    if c["HI"]:
        parts += [("q_I", c["HI"], 0, 0, c["d_I"], "half", t), ("k_I", 1, 0, 0, c["d_I"], "half", shared)]
    return parts


def work(case):
    c = case
    if c["op"] == "rope":
        n, moved, flops = c["n_tok"], 0, 0
        for _, H, _, _, dim, _, t in _parts(c):
            moved += 2 * n * H * (dim or c["rot"]) * _SIZE[t]
            flops += 3 * n * H * c["rot"]  # four products and two sums for a pair
        return {"bytes": moved + 4 * n, "flops": flops}
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * _SIZE[c["dtype"]] + 12 * c["rows"], "flops": n if c["mode"] == "greedy" else 3 * n}
    counts = _counts(c)
    words = -(-max(counts) // 64) if c["tree"] else 0
    return {"bytes": sum(counts) * (16 + 8 * words) + 12 * len(counts), "flops": 0}


def _counts(c):
    rng = random.Random(c["pick"])
    return [rng.randint(c["lo"], c["hi"]) for _ in range(c["n_seqs"])]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = globals()["_prepare_" + case["op"]](case, gen, random.Random(seed))
    s["case"] = case
    return s


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _prepare_rope(c, gen, rng):
    n, s = c["n_tok"], {"x": [], "out": []}
    if c["far"]:  # tokens of several requests, anywhere in their contexts
        s["pos"] = torch.randint(0, c["far"], (n,), dtype=torch.int32, device=DEV, generator=gen)
    else:
        s["pos"] = torch.arange(n, dtype=torch.int32, device=DEV)
    for _, H, before_x, before_out, dim, _, t in _parts(c):
        wide = [(n, H, before + (dim or c["rot"])) for before in (before_x, before_out)]
        x = torch.randn(wide[0], dtype=_TYPE[t], device=DEV, generator=gen)
        out = torch.zeros(wide[1], dtype=_TYPE[t], device=DEV)
        s["x"].append(x[..., before_x:])
        s["out"].append(out[..., before_out:])
    if own:
        import sparse_attention_long_gb300 as dsa
        s["rope"] = dsa.make_rope(
            rot_dim=c["rot"], base=c["base"], scaling=None if c["scaling"] == "none" else c["scaling"],
            factor=c["factor"], original=c["original"], mscale=_mscale(c),
            parts=[dsa.rope_part(heads=H, dim=dim or c["rot"], layout=layout, dtype=t)
                   for _, H, _, _, dim, layout, t in _parts(c)])
    return s


def _mscale(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0


def _prepare_sample(c, gen, rng):
    n, V = c["rows"], c["vocab"]
    logits = torch.randn(n, c["ld"], dtype=torch.float32, device=DEV, generator=gen).mul_(c["spread"])
    # a few tokens that the model thinks likely
    part = V // 12
    at = torch.randint(0, part, (n, 12), device=DEV, generator=gen) + part * torch.arange(12, device=DEV)
    up = 4 * c["spread"] + torch.empty(n, 12, device=DEV).exponential_(0.5, generator=gen)
    logits.scatter_(1, at, up)
    s = dict(logits=logits.to(_TYPE[c["dtype"]]), u=torch.rand(n, device=DEV, generator=gen), index=None,
             temperature=None, top_k=None, top_p=None, min_p=None)
    m, mode = c["requests"] or n, c["mode"]
    if c["requests"]:
        s["index"] = torch.randint(0, m, (n,), device=DEV, generator=gen).sort().values.int()
    reals = lambda lo, hi: torch.tensor([rng.uniform(lo, hi) for _ in range(m)], dtype=torch.float32, device=DEV)
    if mode == "greedy":
        s["temperature"] = torch.zeros(m, device=DEV)
    else:
        s["temperature"] = reals(0.6, 1.2)
    if mode == "usual":
        s["top_k"], s["top_p"] = _ints([_log(rng, 10, 100) for _ in range(m)]), reals(0.8, 0.98)
    elif mode == "nucleus":
        s["top_p"] = reals(0.8, 0.98)
    elif mode == "mixed":  # 0 and 1: that request does without
        some = lambda x, off: x if rng.random() < 0.5 else off
        s["temperature"] = s["temperature"] * _ints([some(1, some(1, 0)) for _ in range(m)])
        s["top_k"] = _ints([some(_log(rng, 1, 2000), 0) for _ in range(m)])
        s["top_p"] = torch.tensor([some(rng.uniform(0.5, 0.99), 1.0) for _ in range(m)], device=DEV)
        s["min_p"] = torch.tensor([some(rng.uniform(0.001, 0.2), 0.0) for _ in range(m)], device=DEV)
    s.update(token=torch.zeros(n, dtype=torch.int32, device=DEV), prob=torch.zeros(n, device=DEV))
    if own:
        import sparse_attention_long_gb300 as dsa
        s["sampler"] = dsa.make_sampler(rows=n, vocab=V, ld=c["ld"], dtype=c["dtype"], requests=c["requests"] or None)
    return s


def _prepare_accept(c, gen, rng):
    counts = _counts(c)
    words = -(-max(counts) // 64)
    masks, drafted, sampled = [], [], []
    for T in counts:
        rows, at = [], len(sampled)
        sampled += [rng.randrange(32000) for _ in range(T)]
        taken = set()
        for t in range(T):
            p = rng.randrange(t) if c["tree"] and t else t - 1
            rows.append((1 << t) | (rows[p] if t else 0))
            hit = t > 0 and p not in taken and rng.random() < c["match"]
            if hit:
                taken.add(p)
            drafted.append(sampled[at + p] if hit else rng.randrange(32000))
        masks += rows
    total = len(sampled)
    # the program may leave room behind the last sequence's tokens; this one has none
    starts = [0]
    for T in counts:
        starts.append(starts[-1] + T)
    s = dict(counts=counts, widest=max(counts), tok_start=_ints(starts), drafted=_ints(drafted), sampled=_ints(sampled),
             mask=None, n_new=_ints([0] * c["n_seqs"]), row_index=_ints([0] * total), tokens=_ints([0] * total),
             next=_ints([0] * c["n_seqs"]))
    if c["tree"]:
        w64 = [[(m >> (64 * w)) & ((1 << 64) - 1) for w in range(words)] for m in masks]
        s["mask"] = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in w64], dtype=torch.int64,
                                 device=DEV)
    if own:
        import sparse_attention_long_gb300 as dsa
        s["cache"] = dsa.make_cache(n_seqs=c["n_seqs"], n_pages=1, page_rows=64, max_pages=1)
        s["attn"] = dsa.make_tree(n_tok=total, H=128, d_qk=576, d_v=512, scale=1.0, mask_words=words if c["tree"] else 0)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _own_rope(s):
    import sparse_attention_long_gb300 as dsa
    dsa.rope_apply(s["rope"], s["pos"], s["x"], s["out"], transposed=s["case"]["back"])
    return s["out"]


def _frequencies(c):
    """Angle per position of each pair."""
    r, base = c["rot"], c["base"]
    if c["scaling"] == "ntk":
        base = base * c["factor"] ** (r / (r - 2)) if r > 2 else base
    plain = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if c["scaling"] == "linear":
        return [f / c["factor"] for f in plain]
    if c["scaling"] != "yarn":
        return plain
    # pairs that turn often keep their frequency, those that turn less than once are stretched
    where = lambda turns: r * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(where(32.0)), 0), min(math.ceil(where(1.0)), r - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(r // 2)]
    return [f * (1 - g) + f / c["factor"] * g for f, g in zip(plain, ramp)]


def _plain_rope(s):
    c = s["case"]
    r = c["rot"]
    # 64 bits: a far position times a frequency has few bits left for the fraction of a turn
    angle = s["pos"].double()[:, None] * torch.tensor(_frequencies(c), dtype=torch.float64, device=DEV)
    cos, sin = (_mscale(c) * angle.cos()).float()[:, None], (_mscale(c) * angle.sin()).float()[:, None]
    sin = -sin if c["back"] else sin
    return [_turned(x, r, cos, sin, layout) for x, (_, _, _, _, _, layout, _) in zip(s["x"], _parts(c))]


def _turned(x, r, cos, sin, layout):
    y = x[..., :r].float()
    if layout == "half":
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y.to(x.dtype), x[..., r:]], -1) if r < x.shape[-1] else y.to(x.dtype)


def _own_sample(s):
    import sparse_attention_long_gb300 as dsa
    dsa.sample(s["sampler"], s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["index"],
               s["token"], s["prob"])
    return {"token": s["token"], "prob": s["prob"]}


def _plain_sample(s):
    V = s["case"]["vocab"]
    # 64 bits: with a large vocabulary a border between two tokens is always near
    x = s["logits"][:, :V].double()
    of = lambda t: (t if s["index"] is None else t[s["index"].long()])[:, None]
    T = of(s["temperature"]).double()
    top = x.amax(-1, keepdim=True)
    ordered, at = torch.sort(x, dim=-1, descending=True, stable=True)
    w = torch.exp((ordered - top) / torch.where(T > 0, T, 1.0))
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["min_p"] is not None:
        keep &= w >= of(s["min_p"]).double()
    rank = torch.arange(V, device=DEV)
    if s["top_k"] is not None:
        k = of(s["top_k"])
        keep &= rank < torch.where(k > 0, k, V)
    if s["top_p"] is not None:
        p = of(s["top_p"]).double()
        mass = torch.cumsum(w * keep, -1)
        before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], -1)
        keep &= (before < p * mass[:, -1:]) | (p >= 1)
    keep = torch.where(T > 0, keep, rank < 1)
    # back in the order of the tokens
    w = torch.zeros_like(w).scatter_(1, at, w * keep)
    mass = torch.cumsum(w, -1)
    target = s["u"].double()[:, None] * mass[:, -1:]
    token = (mass <= target).sum(-1, keepdim=True)
    prob = torch.gather(w, 1, token) / mass[:, -1:]
    return {"token": token[:, 0].int(), "prob": prob[:, 0].float()}


def _own_accept(s):
    import sparse_attention_long_gb300 as dsa
    dsa.tree_accept(s["cache"], s["attn"], s["tok_start"], s["mask"], s["drafted"], s["sampled"], s["n_new"],
                    s["row_index"], s["tokens"], s["next"])
    return {"n_new": s["n_new"], "row_index": s["row_index"], "tokens": s["tokens"], "next": s["next"]}


def _plain_accept(s):
    n, W = s["case"]["n_seqs"], s["widest"]
    start = s["tok_start"].long()
    t = torch.arange(W, device=DEV)
    there = t[None] < (start[1:] - start[:-1])[:, None]
    row = torch.where(there, start[:-1, None] + t[None], 0)
    if s["mask"] is None:
        seen = (t[None, :] <= t[:, None]).expand(n, W, W)
    else:
        bits = (s["mask"][row][..., None] >> torch.arange(64, device=DEV)) & 1
        seen = bits.flatten(-2)[..., :W].bool()
    parent = torch.where(seen & (t[None, :] < t[:, None]), t, -1).amax(-1)
    drafted, sampled = s["drafted"][row], s["sampled"][row]
    good = (parent >= 0) & (drafted == torch.gather(sampled, 1, parent.clamp(min=0)))
    # of several children with the same token the first
    twin = (parent[:, :, None] == parent[:, None, :]) & good[:, None, :] & (t[None, :] < t[:, None])
    good = (good & ~twin.any(-1)) | (t == 0)
    ok = (~seen | good[:, None, :]).all(-1) & seen[:, :, 0] & there
    count = ok.sum(-1)
    place = torch.where(ok, torch.cumsum(count, 0)[:, None] - count[:, None] + torch.cumsum(ok, -1) - 1, row.max() + 1)
    room = torch.full((s["drafted"].numel() + 1,), -1, dtype=torch.int32, device=DEV)
    row_index = room.clone().scatter_(0, place.flatten(), row.flatten().int())[:-1]
    tokens = room.scatter_(0, place.flatten(), sampled.flatten())[:-1]
    last = torch.where(ok, t, -1).amax(-1)
    nxt = torch.where(last >= 0, torch.gather(sampled, 1, last.clamp(min=0)[:, None])[:, 0], -1)
    return {"n_new": count.int(), "row_index": row_index, "tokens": tokens, "next": nxt.int()}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "rope":
        return _exact_rope(case, prepare(case, seed))
    if case["op"] == "sample":
        return _exact_sample(case, prepare(case, seed))
    return None  # whole numbers


def _exact_rope(c, s):
    """Products of complex numbers, pair by pair; the angle is reduced to one turn before its sine is taken."""
    r = c["rot"]
    outs = []
    for x, (_, _, _, _, _, layout, _) in zip(s["x"], _parts(c)):
        y = x.double().clone()
        for i in range(r // 2):
            base = c["base"] * (c["factor"] ** (r / (r - 2.0)) if c["scaling"] == "ntk" and r > 2 else 1.0)
            f = math.exp(-2.0 * i / r * math.log(base))
            if c["scaling"] == "linear":
                f /= c["factor"]
            if c["scaling"] == "yarn":
                lo = r * math.log(c["original"] / (64 * math.pi)) / (2 * math.log(c["base"]))
                hi = r * math.log(c["original"] / (2 * math.pi)) / (2 * math.log(c["base"]))
                lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), r - 1)
                part = 0.0 if i <= lo else 1.0 if i >= hi else (i - lo) / (hi - lo)
                f = f / c["factor"] * part + f * (1 - part)
            turn = torch.polar(torch.full_like(s["pos"], 1, dtype=torch.float64),
                               torch.remainder(s["pos"].double() * f, 2 * math.pi))
            if c["scaling"] == "yarn":
                turn = turn * (1 + math.log(c["factor"]) / 10)
            j, k = (i, i + r // 2) if layout == "half" else (2 * i, 2 * i + 1)
            z = torch.complex(x[..., j].double(), x[..., k].double()) * (turn.conj() if c["back"] else turn)[:, None]
            y[..., j], y[..., k] = z.real, z.imag
        outs.append(y)
    return outs


def _exact_sample(c, s):
    """Row by row; the kept tokens are found from the largest logit downwards."""
    tokens, probs = [], []
    get = lambda t, i: None if t is None else float(t[i])
    rows = s["index"].tolist() if s["index"] is not None else range(c["rows"])
    host = {k: (None if s[k] is None else s[k].tolist()) for k in ("temperature", "top_k", "top_p", "min_p")}
    for i, q in enumerate(rows):
        x = s["logits"][i, :c["vocab"]].double()
        T, k, p, least = (get(host[n], q) for n in ("temperature", "top_k", "top_p", "min_p"))
        if T == 0:
            tokens.append(torch.nonzero(x == x.max())[0, 0])
            probs.append(torch.ones((), dtype=torch.float64, device=DEV))
            continue
        logw = (x - x.max()) / T
        n = c["vocab"] if not least else int((logw >= math.log(least)).sum())
        if k:
            n = min(n, int(k))
        order = torch.argsort(x, descending=True, stable=True)[:n]
        mass = logw[order].exp().cumsum(0)
        if p is not None and p < 1:
            n = 1 + int((mass[:-1] < p * mass[-1]).sum())
        kept = order[:n].sort().values
        share = logw[kept].exp()
        share = share / share.sum()
        j = torch.searchsorted(share.cumsum(0), s["u"][i].double(), right=True).clamp(max=n - 1)
        tokens.append(kept[j])
        probs.append(share[j])
    return {"token": torch.stack(tokens).int(), "prob": torch.stack(probs)}
