"""Measured cases of the decoding operators: attention of drafted tokens over a
paged cache, beam selection, and the page bookkeeping between two steps.

``run`` computes an operator in its plain form (elementary torch operations) or,
with ``own`` true, through the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
LATENT = dict(d_qk=576, d_v=512, scale=1.0 / math.sqrt(192.0), dtype="bf16")
TINY = dict(d_qk=80, d_v=64, scale=1.0 / math.sqrt(80.0), dtype="fp32")


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # attention of drafted tokens over a paged latent cache
        # one user, one new token, a short chat: latency
        dict(name="tree-one", op="tree", n_seqs=1, lo=1023, hi=1023, T=1, H=128, R=64, tree=False, pick=1,
             **LATENT),
        # a serving batch of single tokens, contexts of every length
        dict(name="tree-decode", op="tree", n_seqs=64, lo=517, hi=16384, T=1, H=128, R=64, tree=False, pick=2,
             **LATENT),
        # the same batch size with a drafted tree per sequence
        dict(name="tree-draft", op="tree", n_seqs=16, lo=1900, hi=6144, T=48, H=128, R=64, tree=True, pick=3,
             **LATENT),
        # two long documents on one tensor-parallel shard of the heads, a chain of drafts
        dict(name="tree-long", op="tree", n_seqs=2, lo=60001, hi=65536, T=33, H=16, R=128, tree=False, pick=4,
             **LATENT),
        # the exact path on the small fp32 shapes
        dict(name="tree-fp32", op="tree", n_seqs=5, lo=1, hi=700, T=7, H=8, R=16, tree=True, pick=5, **TINY),
        # beam selection
        # one request, four beams, a small vocabulary of odd size: latency
        dict(name="beam-one", op="beam", n_batch=1, beams=4, keep=4, vocab=32001, ld=32001, dtype="fp32",
             fresh=False),
        # a batch on a large vocabulary, logits rows padded to whole lines
        dict(name="beam-batch", op="beam", n_batch=64, beams=8, keep=8, vocab=131071, ld=131072, dtype="bf16",
             fresh=False),
        # a beam-search step of the cache: fork by parents, copy the shared
        # tails, one new row per beam and layer
        dict(name="step-one", op="step", n_batch=1, beams=4, keep_parents=False, lo=1000, hi=1000, new=1, layers=2,
             R=64, D=576, dtype="bf16", pick=6),
        dict(name="step-beams", op="step", n_batch=32, beams=8, keep_parents=False, lo=1024, hi=4096, new=1,
             layers=8, R=64, D=576, dtype="bf16", pick=7),
        # a serving step after speculative decoding: up to 4 accepted rows of
        # FP8 index keys with their scale, no fork
        dict(name="step-accept", op="step", n_batch=128, beams=1, keep_parents=True, lo=300, hi=16000, new=4,
             layers=16, R=64, D=132, dtype="u8", pick=8),
        # compaction of a fragmented pool
        dict(name="compact-small", op="compact", n_seqs=16, n_pages=512, live=0.5, layers=1, R=64, D=576,
             dtype="bf16", pick=9),
        dict(name="compact-large", op="compact", n_seqs=192, n_pages=16384, live=0.6, layers=1, R=64, D=576,
             dtype="bf16", pick=10),
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
        op = rng.choice(["tree", "tree", "beam", "step", "compact"])
        pick = rng.randrange(1 << 30)
        if op == "tree":
            if rng.random() < 0.2:
                c = dict(op=op, n_seqs=_log(rng, 1, 8), T=_log(rng, 1, 16), H=rng.choice([1, 4, 8, 12]),
                         R=rng.choice([1, 16, 24, 64]), tree=rng.random() < 0.5, **TINY)
                top = 1500
            else:
                c = dict(op=op, n_seqs=_log(rng, 1, 64), T=_log(rng, 1, 100), H=rng.choice([8, 16, 24, 32, 64, 128, 128]),
                         R=rng.choice([16, 32, 64, 64, 128, 256]), tree=rng.random() < 0.5, **LATENT)
                top = 131072
            hi = _log(rng, 16, top)
            c.update(lo=rng.randrange(0, hi), hi=hi, pick=pick)
        elif op == "beam":
            beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
            vocab = _log(rng, 1000, 200000)
            c = dict(op=op, n_batch=_log(rng, 1, 128), beams=beams, keep=rng.choice([beams, rng.randrange(1, 33)]),
                     vocab=vocab, ld=vocab if rng.random() < 0.5 else (vocab + 63) // 64 * 64,
                     dtype=rng.choice(["fp32", "bf16"]), fresh=rng.random() < 0.2)
        elif op == "step":
            D, dtype = rng.choice([(576, "bf16"), (128, "bf16"), (132, "u8"), (128, "u8"), (80, "fp32"), (577, "u8")])
            hi = _log(rng, 64, 16384)
            c = dict(op=op, n_batch=_log(rng, 1, 64), beams=rng.choice([1, 2, 4, 8, 16]),
                     keep_parents=rng.random() < 0.3, lo=rng.randrange(0, hi), hi=hi, new=rng.randrange(1, 9),
                     layers=_log(rng, 1, 16), R=rng.choice([1, 16, 48, 64, 128]), D=D, dtype=dtype, pick=pick)
        else:
            D, dtype = rng.choice([(576, "bf16"), (128, "bf16"), (132, "u8"), (80, "fp32")])
            c = dict(op=op, n_seqs=_log(rng, 1, 256), n_pages=_log(rng, 16, 16384), live=rng.uniform(0.05, 0.95),
                     layers=_log(rng, 1, 4), R=rng.choice([16, 48, 64, 128]), D=D, dtype=dtype, pick=pick)
        if op in ("step", "compact") and _pool_bytes(c) > 6 << 30:
            continue
        w = work(c)
        if w["bytes"] <= largest[op][0] and w["flops"] <= largest[op][1]:
            return c


def _lens(c, n):
    rng = random.Random(c["pick"])
    return [rng.randint(c["lo"], c["hi"]) for _ in range(n)]


def _cdiv(a, b):
    return -(-a // b)


def _tree_masks(c):
    """Per sequence, per drafted token: the set of drafted tokens it sees, as an integer of bits."""
    rng = random.Random(c["pick"] + 1)
    out = []
    for _ in range(c["n_seqs"]):
        rows = []
        for t in range(c["T"]):
            seen = 1 << t
            if t and rng.random() > 0.1:  # a child of an earlier token, else another root
                seen |= rows[rng.randrange(t)] if c["tree"] else rows[t - 1]
            elif t and not c["tree"]:
                seen |= rows[t - 1]
            rows.append(seen)
        out.append(rows)
    return out


_SIZE = {"bf16": 2, "fp32": 4, "u8": 1}
_TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32, "u8": torch.uint8}


def work(case):
    c = case
    if c["op"] == "tree":
        e = _SIZE[c["dtype"]]
        lens = _lens(c, c["n_seqs"])
        n_tok = c["T"] * c["n_seqs"]
        if c["tree"]:
            drafted = sum(bin(m).count("1") for rows in _tree_masks(c) for m in rows)
        else:
            drafted = c["n_seqs"] * c["T"] * (c["T"] + 1) // 2
        keys = sum(lens) * c["T"] + drafted
        return {"bytes": (sum(lens) + n_tok) * c["d_qk"] * e + n_tok * c["H"] * ((c["d_qk"] + c["d_v"]) * e + 8),
                "flops": 2 * keys * c["H"] * (c["d_qk"] + c["d_v"])}
    if c["op"] == "beam":
        n = c["n_batch"] * c["beams"] * c["vocab"]
        # a subtraction, an exponential and a sum for each logit
        return {"bytes": n * _SIZE[c["dtype"]] + c["n_batch"] * (5 * c["beams"] + 13 * c["keep"]), "flops": 3 * n}
    row = c["D"] * _SIZE[c["dtype"]] * c["layers"]
    if c["op"] == "step":
        p = _step_plan(c)
        entries = sum(_cdiv(n, c["R"]) for n in p["lens"])
        rows = 2 * p["copied_rows"] + 2 * sum(p["n_new"])  # each read once and written once
        return {"bytes": rows * row + 8 * entries + 8 * p["n_pages"], "flops": 0}
    p = _compact_plan(c)
    return {"bytes": 2 * len(p["moves"]) * c["R"] * row + 8 * sum(p["pages"]) + 12 * c["n_pages"], "flops": 0}


# --------------------------------------------------------------------------
# plans of the cache cases (host side, from the case alone)
# --------------------------------------------------------------------------
def _step_plan(c):
    rng = random.Random(c["pick"] + 2)
    base = _lens(c, c["n_batch"])
    R, W = c["R"], c["beams"]
    lens = [n for n in base for _ in range(W)]
    parents, copied, dup = [], 0, 0
    for b in range(c["n_batch"]):
        mine = [b * W + (w if c["keep_parents"] else rng.randrange(W)) for w in range(W)]
        again = W - len(set(mine))
        if base[b] % R:
            copied += again * (base[b] % R)
            dup += again
        parents += mine
    n_new = [rng.randint(1, c["new"]) for _ in lens]
    # the beams of a request share their first pages
    shared = [int(0.9 * (n // R)) for n in base]
    used = sum(s + W * (_cdiv(n, R) - s) for n, s in zip(base, shared))
    grown = sum(_cdiv(n + a, R) - _cdiv(n, R) for n, a in zip(lens, n_new))
    n_pages = used + dup + grown + len(lens) + 8
    return dict(lens=lens, base=base, parents=parents, n_new=n_new, shared=shared, n_pages=n_pages,
                copied_rows=copied, dup=dup, max_pages=_cdiv(max(lens) + c["new"], R) + 1)


def _compact_plan(c):
    rng = random.Random(c["pick"] + 3)
    n_live = max(1, int(c["live"] * c["n_pages"]))
    ids = list(range(c["n_pages"]))
    rng.shuffle(ids)
    live = ids[:n_live]
    n = min(c["n_seqs"], n_live)
    cuts = [0] + sorted(rng.sample(range(1, n_live), n - 1)) + [n_live] if n > 1 else [0, n_live]
    owned = [live[a:b] for a, b in zip(cuts, cuts[1:])] + [[] for _ in range(c["n_seqs"] - n)]
    is_live = [False] * c["n_pages"]
    for p in live:
        is_live[p] = True
    holes = [p for p in range(n_live) if not is_live[p]]
    movers = [p for p in range(n_live, c["n_pages"]) if is_live[p]]
    return dict(owned=owned, n_live=n_live, moves=list(zip(movers, holes)), pages=[len(o) for o in owned])


def _pool_bytes(c):
    n = _step_plan(c)["n_pages"] if c["op"] == "step" else c["n_pages"]
    return n * c["R"] * c["D"] * _SIZE[c["dtype"]] * c["layers"]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _values(shape, dtype, gen, scale=1.0):
    if dtype == "u8":
        return torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen)
    t = torch.randn(shape, dtype=_TYPE[dtype], device=DEV, generator=gen)
    return t.mul_(scale) if scale != 1.0 else t


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = globals()["_prepare_" + c["op"]](c, gen, random.Random(seed))
    s["case"] = c
    return s


def _prepare_tree(c, gen, rng):
    n, R, T, H = c["n_seqs"], c["R"], c["T"], c["H"]
    lens = _lens(c, n)
    pages = [_cdiv(x, R) for x in lens]
    n_pages = max(1, sum(pages) + sum(pages) // 8)
    max_pages = max(1, max(pages))
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, at = [], 0
    for p in pages:
        table.append(ids[at:at + p] + [-1] * (max_pages - p))
        at += p
    sc = 1.0 if c["dtype"] == "bf16" else c["d_qk"] ** -0.5
    n_tok = n * T
    s = dict(pool=_values((n_pages, R, c["d_qk"]), c["dtype"], gen, sc),
             q=_values((n_tok, H, c["d_qk"]), c["dtype"], gen, sc),
             kv_new=_values((n_tok, c["d_qk"]), c["dtype"], gen, sc),
             table=_ints(table), lens=_ints(lens), tok_start=_ints([T * i for i in range(n + 1)]),
             host_lens=lens, mask=None)
    words = _cdiv(T, 64)
    masks = _tree_masks(c)
    if c["tree"]:
        w64 = [[(m >> (64 * w)) & ((1 << 64) - 1) for w in range(words)] for rows in masks for m in rows]
        s["mask"] = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in w64], dtype=torch.int64,
                                 device=DEV)
    # the same visibility as truth values [sequence, token, drafted key], for the plain form
    s["seen"] = torch.tensor([[[(m >> j) & 1 for j in range(T)] for m in rows] for rows in masks], dtype=torch.bool,
                             device=DEV)
    dt = _TYPE[c["dtype"]]
    s.update(out=torch.zeros(n_tok, H, c["d_v"], dtype=dt, device=DEV), m=torch.zeros(n_tok, H, device=DEV),
             l=torch.zeros(n_tok, H, device=DEV))
    if own:
        import sparse_attention_long_gb300 as dsa
        s["cache"] = dsa.make_cache(n_seqs=n, n_pages=n_pages, page_rows=R, max_pages=max_pages)
        s["attn"] = dsa.make_tree(n_tok=n_tok, H=H, d_qk=c["d_qk"], d_v=c["d_v"], scale=c["scale"], dtype=c["dtype"],
                                  mask_words=words if c["tree"] else 0)
        s["ws"] = torch.empty(dsa.tree_workspace_size(s["cache"], s["attn"]), dtype=torch.uint8, device=DEV)
    return s


def _prepare_beam(c, gen, rng):
    n, W, V = c["n_batch"], c["beams"], c["vocab"]
    logits = _values((n, W, c["ld"]), c["dtype"], gen, 2.5)
    scores = -20.0 * torch.rand(n, W, device=DEV, generator=gen)
    finished = torch.rand(n, W, device=DEV, generator=gen) < 0.1
    if c["fresh"]:  # the first step: one beam of each request is alive
        scores.fill_(-math.inf)
        scores[:, 0] = 0.0
        finished.fill_(False)
    s = dict(logits=logits, scores=scores, finished=finished.to(torch.uint8), eos=min(2, V - 1))
    s.update(parent=torch.zeros(n, c["keep"], dtype=torch.int32, device=DEV),
             token=torch.zeros(n, c["keep"], dtype=torch.int32, device=DEV),
             scores_out=torch.zeros(n, c["keep"], device=DEV),
             finished_out=torch.zeros(n, c["keep"], dtype=torch.uint8, device=DEV))
    if own:
        import sparse_attention_long_gb300 as dsa
        s["beam"] = dsa.make_beam(n_batch=n, beams_in=W, beams_out=c["keep"], vocab=V, ld=c["ld"], dtype=c["dtype"],
                                  eos=s["eos"])
        s["ws"] = torch.empty(dsa.beam_workspace_size(s["beam"]), dtype=torch.uint8, device=DEV)
    return s


def _prepare_step(c, gen, rng):
    p = _step_plan(c)
    R, W, n = c["R"], c["beams"], len(p["lens"])
    ids = list(range(p["n_pages"]))
    rng.shuffle(ids)
    table, refs, at = [], [0] * p["n_pages"], 0
    for b, length in enumerate(p["base"]):
        first = ids[at:at + p["shared"][b]]
        at += len(first)
        for _ in range(W):
            own_pages = _cdiv(length, R) - len(first)
            row = first + ids[at:at + own_pages]
            at += own_pages
            for x in row:
                refs[x] += 1
            table.append(row + [-1] * (p["max_pages"] - len(row)))
    cap = n * c["new"]
    pool = _values((c["layers"], p["n_pages"], R, c["D"]), c["dtype"], gen)
    s = dict(pool=pool, rows=_values((c["layers"], cap, c["D"]), c["dtype"], gen), table=_ints(table),
             lens=_ints(p["lens"]), refs=_ints(refs), parent=_ints(p["parents"]), n_new=_ints(p["n_new"]),
             dup=p["dup"], total=sum(p["n_new"]), max_pages=p["max_pages"],
             table_out=torch.zeros(n, p["max_pages"], dtype=torch.int32, device=DEV),
             lens_out=torch.zeros(n, dtype=torch.int32, device=DEV),
             refs_out=torch.zeros(p["n_pages"], dtype=torch.int32, device=DEV),
             copies=torch.zeros(n, 3, dtype=torch.int32, device=DEV),
             n_copies=torch.zeros(1, dtype=torch.int32, device=DEV),
             slots=torch.zeros(cap, dtype=torch.int32, device=DEV))
    if own:
        import sparse_attention_long_gb300 as dsa
        s["cache"] = dsa.make_cache(n_seqs=n, n_pages=p["n_pages"], page_rows=R, max_pages=p["max_pages"])
    return s


def _prepare_compact(c, gen, rng):
    p = _compact_plan(c)
    R, n, n_pages = c["R"], c["n_seqs"], c["n_pages"]
    max_pages = max(p["pages"])
    refs = [0] * n_pages
    for o in p["owned"]:
        for x in o:
            refs[x] += 1
    lens = [len(o) * R - (rng.randrange(R) if o else 0) for o in p["owned"]]
    s = dict(pool=_values((c["layers"], n_pages, R, c["D"]), c["dtype"], gen),
             table=_ints([o + [-1] * (max_pages - len(o)) for o in p["owned"]]), lens=_ints(lens), refs=_ints(refs),
             n_moves=len(p["moves"]),
             table_out=torch.zeros(n, max_pages, dtype=torch.int32, device=DEV),
             refs_out=torch.zeros(n_pages, dtype=torch.int32, device=DEV),
             page_map=torch.zeros(n_pages, dtype=torch.int32, device=DEV),
             copies=torch.zeros(n_pages // 2 + 1, 3, dtype=torch.int32, device=DEV),
             n_copies=torch.zeros(1, dtype=torch.int32, device=DEV))
    if own:
        import sparse_attention_long_gb300 as dsa
        s["cache"] = dsa.make_cache(n_seqs=n, n_pages=n_pages, page_rows=R, max_pages=max_pages)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _own_tree(s):
    import sparse_attention_long_gb300 as dsa
    dsa.tree_attn_fwd(s["cache"], s["attn"], s["q"], s["pool"], s["table"], s["lens"], s["kv_new"], s["tok_start"],
                      s["mask"], s["out"], s["m"], s["l"], s["ws"])
    return {"out": s["out"], "softmax_max": s["m"], "softmax_sum": s["l"]}


def _plain_tree(s):
    c = s["case"]
    R, T = c["R"], c["T"]
    for b, n in enumerate(s["host_lens"]):
        t = slice(b * T, (b + 1) * T)
        rows = s["pool"][s["table"][b, :_cdiv(n, R)].long()].reshape(-1, c["d_qk"])[:n]
        k = torch.cat([rows, s["kv_new"][t]]).float()
        x = torch.matmul(s["q"][t].float(), k.T) * c["scale"]
        x[:, :, n:].masked_fill_(~s["seen"][b][:, None, :], -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        l = e.sum(-1, keepdim=True)
        s["out"][t] = (torch.matmul(e, k[:, :c["d_v"]]) / l).to(s["out"].dtype)
        s["m"][t], s["l"][t] = m[..., 0], l[..., 0]
    return {"out": s["out"], "softmax_max": s["m"], "softmax_sum": s["l"]}


def _own_beam(s):
    import sparse_attention_long_gb300 as dsa
    dsa.beam_select(s["beam"], s["logits"], s["scores"], s["finished"], s["parent"], s["token"], s["scores_out"],
                    s["finished_out"], s["ws"])
    return {"parent": s["parent"], "token": s["token"], "scores": s["scores_out"], "finished": s["finished_out"]}


def _plain_beam(s):
    c = s["case"]
    V, W = c["vocab"], c["beams"]
    # 64 bits: candidates of different beams may lie next to each other
    x = s["logits"][..., :V].double()
    top = x.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    cand = s["scores"].double()[..., None] + (x - lse)
    done = s["finished"].bool()
    cand.masked_fill_(done[..., None], -math.inf)
    cand[..., s["eos"]] = torch.where(done, s["scores"].double(), cand[..., s["eos"]])
    best, at = torch.sort(cand.reshape(c["n_batch"], W * V), dim=-1, descending=True, stable=True)
    best, at = best[:, :c["keep"]], at[:, :c["keep"]]
    none = best == -math.inf
    beam, token = at // V, at % V
    first = torch.arange(c["n_batch"], device=DEV)[:, None] * W
    s["parent"].copy_(torch.where(none, -1, first + beam))
    s["token"].copy_(torch.where(none, -1, token))
    s["scores_out"].copy_(best)
    s["finished_out"].copy_((torch.gather(done, 1, beam) | (token == s["eos"])) & ~none)
    return {"parent": s["parent"], "token": s["token"], "scores": s["scores_out"], "finished": s["finished_out"]}


def _own_step(s):
    import sparse_attention_long_gb300 as dsa
    dsa.cache_fork(s["cache"], s["parent"], s["table"], s["lens"], s["refs"], s["table_out"], s["lens_out"],
                   s["refs_out"], s["copies"], s["n_copies"])
    dsa.cache_copy_pages(s["cache"], s["pool"], s["copies"], s["n_copies"])
    dsa.cache_extend(s["cache"], s["n_new"], s["table_out"], s["lens_out"], s["refs_out"], s["lens_out"],
                     s["refs_out"], s["slots"])
    dsa.cache_write(s["cache"], s["pool"], s["rows"], s["slots"])
    return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"], "slots": s["slots"],
            "pool": s["pool"]}


def _free_pages(refs):
    return torch.argsort((refs > 0).to(torch.uint8), stable=True)  # the free ones first, ascending


def _held(lens, R, max_pages):
    return torch.arange(max_pages, device=DEV)[None, :] < ((lens + R - 1) // R)[:, None]


def _plain_step(s):
    c = s["case"]
    R, n, P = c["R"], s["lens"].numel(), s["refs"].numel()
    at = torch.arange(n, device=DEV)
    par = s["parent"].long()
    # fork: page references follow the parents; the first child of a parent
    # keeps its partial last page, the others get a copy in the lowest free pages
    lens = s["lens"][par]
    table = torch.where(_held(lens, R, s["max_pages"]), s["table"][par], -1)
    first = torch.full((n,), n, device=DEV).scatter_reduce_(0, par, at, "amin")
    need = (first[par] != at) & (lens % R != 0)
    last = (lens // R).clamp(max=s["max_pages"] - 1).long()
    kept = _held(lens, R, s["max_pages"])
    kept[at, last] &= ~need
    refs = torch.zeros(P + 1, dtype=torch.int32, device=DEV)
    refs.index_add_(0, torch.where(kept, table, P).reshape(-1).long(),
                    torch.ones(table.numel(), dtype=torch.int32, device=DEV))
    refs = refs[:P]
    who = torch.argsort((~need).to(torch.uint8), stable=True)[:s["dup"]]
    dst = _free_pages(refs)[:s["dup"]]
    src = table[who, last[who]].long()
    rows = (torch.arange(R, device=DEV)[None, :] < (lens[who] % R)[:, None])[None, :, :, None]
    s["pool"][:, dst] = torch.where(rows, s["pool"][:, src], s["pool"][:, dst])
    table[who, last[who]] = dst.int()
    refs[dst] = 1
    # extend: further pages in the order of the sequences, lowest free first
    now = (lens + R - 1) // R
    more = (lens + s["n_new"] + R - 1) // R - now
    begin = torch.cumsum(more, 0) - more
    free = _free_pages(refs)
    for j in range(_cdiv(c["new"], R) + 1):
        got = more > j
        page = free[(begin + j).clamp(max=P - 1).long()]
        col = (now + j).clamp(max=s["max_pages"] - 1).long()
        table[at, col] = torch.where(got, page.int(), table[at, col])
        refs.index_add_(0, page, got.int())
    ends = torch.cumsum(s["n_new"], 0)
    i = torch.arange(s["slots"].numel(), device=DEV)
    seq = torch.searchsorted(ends, i, right=True).clamp(max=n - 1)
    pos = lens[seq] + i - (ends - s["n_new"])[seq]
    ok = i < s["total"]
    pos = torch.where(ok, pos, 0)
    slot = table[seq, (pos // R).long()] * R + pos % R
    s["slots"].copy_(torch.where(ok, slot, -1))
    flat = s["pool"].view(c["layers"], P * R, c["D"])
    flat[:, s["slots"][:s["total"]].long()] = s["rows"][:, :s["total"]]
    s["table_out"].copy_(table)
    s["lens_out"].copy_(lens + s["n_new"])
    s["refs_out"].copy_(refs)
    return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"], "slots": s["slots"],
            "pool": s["pool"]}


def _own_compact(s):
    import sparse_attention_long_gb300 as dsa
    dsa.cache_compact(s["cache"], s["table"], s["lens"], s["refs"], s["table_out"], s["refs_out"], s["page_map"],
                      s["copies"], s["n_copies"])
    dsa.cache_copy_pages(s["cache"], s["pool"], s["copies"], s["n_copies"])
    return {"table": s["table_out"], "refs": s["refs_out"], "map": s["page_map"], "pool": s["pool"]}


def _plain_compact(s):
    c = s["case"]
    P = s["refs"].numel()
    ids = torch.arange(P, device=DEV)
    live = s["refs"] > 0
    n_live = live.sum()
    low = ids < n_live
    holes = torch.argsort((live | ~low).to(torch.uint8), stable=True)
    mover = live & ~low
    rank = (torch.cumsum(mover, 0) - 1).clamp(min=0)
    new = torch.where(mover, holes[rank], ids)
    s["page_map"].copy_(torch.where(live, new, -1))
    src = torch.argsort((~mover).to(torch.uint8), stable=True)[:s["n_moves"]]
    s["pool"][:, holes[:s["n_moves"]]] = s["pool"][:, src]
    held = _held(s["lens"], c["R"], s["table"].shape[1])
    s["table_out"].copy_(torch.where(held, s["page_map"][s["table"].clamp(min=0).long()], -1))
    s["refs_out"].zero_()
    s["refs_out"][:] = torch.where(low, torch.where(live, s["refs"], 0), 0)
    s["refs_out"][holes[:s["n_moves"]]] = s["refs"][src]
    return {"table": s["table_out"], "refs": s["refs_out"], "map": s["page_map"], "pool": s["pool"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "tree":
        return _exact_tree(c, prepare(c, seed))
    if c["op"] == "beam":
        return _exact_beam(c, prepare(c, seed))
    return None  # whole numbers and rows that are moved


def _exact_tree(c, s):
    """One token at a time: softmax over the keys it sees, listed one after the other."""
    if work(c)["flops"] > 2e12:
        return None
    outs, ms, ls = [], [], []
    masks = _tree_masks(c)
    scale = float(torch.tensor(c["scale"], dtype=torch.float32))
    for b, n in enumerate(s["host_lens"]):
        pos = torch.arange(n, device=DEV)
        ids = s["table"][b].long()[pos // c["R"]] if n else pos
        cached = s["pool"][ids, pos % c["R"]].double()
        for t in range(c["T"]):
            seen = [j for j in range(c["T"]) if (masks[b][t] >> j) & 1]
            keys = torch.cat([cached, s["kv_new"][[b * c["T"] + j for j in seen]].double()])
            x = scale * (keys @ s["q"][b * c["T"] + t].double().T)
            m = x.max(0).values
            p = (x - m).exp()
            ls.append(p.sum(0))
            ms.append(m)
            outs.append((p / ls[-1]).T @ keys[:, :c["d_v"]])
    return {"out": torch.stack(outs), "softmax_max": torch.stack(ms), "softmax_sum": torch.stack(ls)}


def _exact_beam(c, s):
    """The best `keep` of each request, from the best `keep` of each beam."""
    rows = []
    for b in range(c["n_batch"]):
        cand = []
        for w in range(c["beams"]):
            if s["finished"][b, w]:
                cand.append(s["scores"][b, w].double()[None])
                continue
            x = s["logits"][b, w, :c["vocab"]].double()
            best = torch.topk(x, min(c["keep"], c["vocab"])).values
            cand.append(s["scores"][b, w].double() + best - torch.logsumexp(x, 0))
        cand = torch.cat(cand)
        cand = torch.cat([cand, torch.full((c["keep"],), -math.inf, dtype=torch.float64, device=DEV)])
        rows.append(torch.topk(cand, c["keep"]).values)
    return {"parent": None, "token": None, "scores": torch.stack(rows), "finished": None}
