"""Paged-cache calls on the GPU against the plain bookkeeping in oracle.cache, exactly."""
import ctypes
import random

import pytest
import torch

from gpu_util import DEV, lib
from oracle import cache as oc

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def random_state(rng, n, R, P, M, dead=0.2):
    """A valid state: shared full pages, own partial ones, spread over the pool."""
    ids = list(range(P))
    rng.shuffle(ids)
    table, lens, refs = [], [], [0] * P
    for i in range(n):
        ln = 0 if rng.random() < dead else rng.randint(1, M * R)
        row = []
        if i and ln:
            j = rng.randrange(i)
            row = table[j][:rng.randint(0, min(lens[j] // R, ln // R))]
        while len(row) < oc.pages_of(ln, R) and ids:
            row = row + [ids.pop()]
        ln = min(ln, len(row) * R)
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (M - len(row)))
        lens.append(ln)
    return table, lens, refs


class Device:
    def __init__(self, dsa, n, R, P, M):
        self.dsa, self.c = dsa, dsa.make_cache(n_seqs=n, n_pages=P, page_rows=R, max_pages=M)
        self.n, self.R, self.P, self.M = n, R, P, M

    def fork(self, parent, table, lens, refs):
        o = [ints([[7] * self.M] * self.n), ints([7] * self.n), ints([7] * self.P), ints([[7] * 3] * self.n), ints([7])]
        self.dsa.cache_fork(self.c, ints(parent), ints(table), ints(lens), ints(refs), *o)
        st = self.dsa.get_status()
        k = int(o[4])
        return [x.tolist() for x in o[:3]] + [[tuple(x) for x in o[3][:k].tolist()]], st

    def extend(self, n_new, table, lens, refs, n_slots, in_place=False):
        t, ln, rf = ints(table), ints(lens), ints(refs)
        lo, ro = (ln, rf) if in_place else (torch.full_like(ln, 7), torch.full_like(rf, 7))
        slots = torch.full((n_slots,), 7, dtype=torch.int32, device=DEV)
        self.dsa.cache_extend(self.c, ints(n_new), t, ln, rf, lo, ro, slots)
        st = self.dsa.get_status()
        return [t.tolist(), lo.tolist(), ro.tolist(), slots.tolist()], st

    def compact(self, table, lens, refs):
        o = [ints([[7] * self.M] * self.n), ints([7] * self.P), ints([7] * self.P),
             ints([[7] * 3] * (self.P // 2 + 1)), ints([7])]
        self.dsa.cache_compact(self.c, ints(table), ints(lens), ints(refs), *o)
        st = self.dsa.get_status()
        k = int(o[4])
        return [x.tolist() for x in o[:3]] + [[tuple(x) for x in o[3][:k].tolist()]], st


def full_table(table, lens, R, M):
    return [row[:oc.pages_of(n, R)] + [-1] * (M - oc.pages_of(n, R)) for row, n in zip(table, lens)]


# one CTA and a cluster; one page row; sizes that do not fill a warp or a slice;
# more sequences and pages than a block has threads
SHAPES = [(1, 1, 1, 1), (1, 16, 5, 3), (5, 3, 33, 7), (33, 4, 700, 20), (64, 64, 2000, 300), (1500, 1, 9000, 4),
          (7, 5, 40001, 5000)]


@pytest.mark.parametrize("n,R,P,M", SHAPES)
@pytest.mark.parametrize("seed", [0, 1])
def test_fork(n, R, P, M, seed):
    rng = random.Random(100 * n + seed)
    d = Device(lib(), n, R, P, M)
    table, lens, refs = random_state(rng, n, R, P // 2 + 1, M)
    refs += [0] * (P - len(refs))
    if P > 3:
        refs[P - 1] += 2  # held by the caller itself
    for parent in ([rng.choice([i, rng.randrange(n), rng.randrange(n), -1]) for i in range(n)], list(range(n)),
                   [-1] * n, [n - 1] * n):
        got, st = d.fork(parent, table, lens, refs)
        want = oc.fork(parent, table, lens, refs, R, M)
        if want is None:  # too few free pages
            assert st == d.dsa.DSA_ERR_PAGES and got == [table, lens, refs, []]
        else:
            assert st == 0 and got == list(want)


@pytest.mark.parametrize("n,R,P,M", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(n, R, P, M, in_place):
    rng = random.Random(n + R)
    d = Device(lib(), n, R, P, M)
    table, lens, refs = random_state(rng, n, R, P // 2 + 1, M)
    refs += [0] * (P - len(refs))
    for most in (0, 1, 3, 2 * R + 1):
        n_new = [rng.randint(0, min(most, M * R - x)) for x in lens]
        for n_slots in (max(1, sum(n_new)), sum(n_new) + 37):
            got, st = d.extend(n_new, table, lens, refs, n_slots, in_place)
            want = oc.extend(n_new, table, lens, refs, R, M, n_slots)
            if want is None:
                assert st in (d.dsa.DSA_ERR_PAGES, d.dsa.DSA_ERR_INDEX)
                assert got == [table, lens, refs, [-1] * n_slots]
            else:
                assert st == 0 and got == list(want)


@pytest.mark.parametrize("n,R,P,M", SHAPES)
def test_compact(n, R, P, M):
    rng = random.Random(n * R)
    d = Device(lib(), n, R, P, M)
    for dead in (0.0, 0.5, 1.0):
        table, lens, refs = random_state(rng, n, R, P, M, dead)
        if P > 3:  # held by the caller: moves, too
            refs[P - 1] += 1
        got, st = d.compact(table, lens, refs)
        assert st == 0 and got == list(oc.compact(table, lens, refs, R, M))


def test_a_call_that_cannot_be_carried_out_changes_nothing():
    R, M, P = 4, 3, 6
    d = Device(lib(), 2, R, P, M)
    table, lens, refs = [[3, 1, -1], [3, -1, -1]], [6, 4], [0, 1, 0, 2, 0, 0]
    E = d.dsa.DSA_ERR_INDEX
    for parent, t, ln in (([2, 0], table, lens), ([-2, 0], table, lens), ([0, 1], [[3, 6, -1], [3, -1, -1]], lens),
                          ([0, 1], [[-1, 1, -1], [3, -1, -1]], lens), ([0, 1], table, [13, 4]), ([0, 1], table, [-1, 4])):
        assert d.fork(parent, t, ln, refs) == ([t, ln, refs, []], E)
    assert d.fork([1, 1], table, lens, [0, 0, 0, 2, 0, 0]) == ([table, lens, [0, 0, 0, 2, 0, 0], []], E)  # refs too low
    for n_new, ln, rf, slots in (([7, 0], lens, refs, 9), ([-1, 0], lens, refs, 9), ([5, 1], lens, refs, 5),
                                 ([1, 0], lens, [0, 2, 0, 2, 0, 0], 5), ([0, 0], [-1, 0], refs, 5),
                                 ([2**31 - 1, 2**31 - 1], lens, refs, 5)):
        assert d.extend(n_new, table, ln, rf, slots) == ([table, ln, rf, [-1] * slots], E)
    full = [1, 1, 1, 2, 1, 1]
    assert d.extend([3, 0], table, lens, full, 5) == ([table, lens, full, [-1] * 5], d.dsa.DSA_ERR_PAGES)
    # old sequence 1 gives up only page 3, which both children still hold: nothing falls free
    assert d.fork([0, 0], table, lens, full) == ([table, lens, full, []], d.dsa.DSA_ERR_PAGES)
    assert d.fork([0, 0], [[3, 1, -1], [2, 4, -1]], [6, 8], [1] * 6) == (
        [[[3, 1, -1], [3, 2, -1]], [6, 6], [1, 1, 1, 2, 0, 1], [(1, 2, 2)]], 0)  # takes a page that falls free
    ident = [p if r else -1 for p, r in enumerate(refs)]
    for t, ln in (([[3, 0, -1], [3, -1, -1]], lens), ([[3, 9, -1], [3, -1, -1]], lens), (table, [13, 4])):
        assert d.compact(t, ln, refs) == ([t, refs, ident, []], E)


KINDS = [((576,), torch.bfloat16), ((132,), torch.uint8), ((7,), torch.uint8), ((80,), torch.float32),
         ((4096,), torch.float32)]


@pytest.mark.parametrize("shape,dtype", KINDS)
@pytest.mark.parametrize("order", ["layers", "pages", "one"])
def test_copies_and_writes_move_the_listed_rows_only(shape, dtype, order):
    dsa = lib()
    L, P, R, D = 3, 9, 5, shape[0]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    make = lambda *s: torch.randint(0, 250, s, device=DEV, generator=gen).to(dtype)
    if order == "layers":
        pool = make(L, P, R, D)
    elif order == "pages":
        pool = make(P, L, R, D).transpose(0, 1)
    else:
        L, pool = 1, make(P, R, D)
    c = dsa.make_cache(n_seqs=1, n_pages=P, page_rows=R, max_pages=2)
    want = pool.clone()
    copies = [(0, 3, 5), (2, 1, 1), (4, 8, 3), (5, 6, 0), (7, 7, 9), (9, 1, 1), (0, -1, 1)]
    w = want if want.dim() == 4 else want[None]
    for s, t, r in copies[:4]:
        w[:, t, :r] = w[:, s, :r]
    dsa.cache_copy_pages(c, pool, ints(copies[:4] + [(1, 2, 5)]), ints([4]))  # the fifth is not counted
    assert dsa.get_status() == 0 and torch.equal(pool, want)
    dsa.cache_copy_pages(c, pool, ints(copies[4:]), ints([50]))               # more than there are; all out of range
    assert dsa.get_status() == dsa.DSA_ERR_INDEX and torch.equal(pool, want)
    dsa.cache_copy_pages(c, pool, ints(copies), ints([-1]))
    assert dsa.get_status() == 0 and torch.equal(pool, want)
    # writes
    n = 6
    rows = make(L, n, D)
    slots = [0, 44, -1, 7, 23, 30]
    flat = w.reshape(L, P * R, D)
    for i, s in enumerate(slots):
        if s >= 0:
            flat[:, s] = rows[:, i]
    w.copy_(flat.view(L, P, R, D))
    dsa.cache_write(c, pool, rows if pool.dim() == 4 else rows[0], ints(slots))
    assert dsa.get_status() == 0 and torch.equal(pool, want)
    pick = [5, 5, 0]
    for s, i in zip([1, 2, 3], pick):
        w[:, s // R, s % R] = rows[:, i]
    dsa.cache_write(c, pool, rows if pool.dim() == 4 else rows[0], ints([1, 2, 3]), ints(pick))
    assert dsa.get_status() == 0 and torch.equal(pool, want)
    for slots, pick in (([45], [0]), ([-2], [0]), ([1], [6]), ([1], [-1])):
        dsa.cache_write(c, pool, rows if pool.dim() == 4 else rows[0], ints(slots), ints(pick))
        assert dsa.get_status() == dsa.DSA_ERR_INDEX and torch.equal(pool, want)


def test_pages_past_four_gigabytes():
    # byte offsets past 2^32 in one layer and between layers
    dsa = lib()
    L, P, R, D = 2, 70000, 64, 576
    pool = torch.zeros(L, P, R, D, dtype=torch.bfloat16, device=DEV)
    c = dsa.make_cache(n_seqs=1, n_pages=P, page_rows=R, max_pages=1)
    rows = torch.randn(L, 2, D, device=DEV).to(torch.bfloat16)
    last = P * R - 1
    dsa.cache_write(c, pool, rows, ints([last, 5 * R + R - 1]))
    dsa.cache_copy_pages(c, pool, ints([[P - 1, 69000, R], [5, P - 2, R]]), ints([2]))
    assert dsa.get_status() == 0
    assert torch.equal(pool[:, P - 1, R - 1], rows[:, 0]) and torch.equal(pool[:, 69000, R - 1], rows[:, 0])
    assert torch.equal(pool[:, P - 2, R - 1], rows[:, 1]) and not pool[:, P - 2, :R - 1].any()
    assert int(pool.count_nonzero(-1).gt(0).sum()) == 2 * 4


def test_run_of_steps_in_a_graph():
    # fork, copy, extend, write captured once and replayed on new inputs, against the plain run
    dsa = lib()
    rng = random.Random(3)
    n, R, P, M, L, D = 6, 4, 80, 10, 2, 16
    d = Device(dsa, n, R, P, M)
    t = [ints([[-1] * M] * n), ints([[-1] * M] * n)]
    ln, rf = [ints([0] * n), ints([0] * n)], [ints([0] * P), ints([0] * P)]
    parent, n_new = ints([0] * n), ints([0] * n)
    copies, k, slots = ints([[0] * 3] * n), ints([0]), ints([0] * 24)
    pool, rows = torch.zeros(L, P, R, D, device=DEV), torch.zeros(L, 24, D, device=DEV)

    def step(a, b):
        dsa.cache_fork(d.c, parent, t[a], ln[a], rf[a], t[b], ln[b], rf[b], copies, k)
        dsa.cache_copy_pages(d.c, pool, copies, k)
        dsa.cache_extend(d.c, n_new, t[b], ln[b], rf[b], ln[b], rf[b], slots)
        dsa.cache_write(d.c, pool, rows, slots)

    side = torch.cuda.Stream()
    graphs = []
    for a, b in ((0, 1), (1, 0)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(a, b)
        graphs.append(g)
    state = ([[-1] * M] * n, [0] * n, [0] * P)
    want = [[] for _ in range(n)]
    for i in range(16):
        par = [rng.choice([j, rng.randrange(n)]) for j in range(n)] if i else list(range(n))
        add = [rng.randrange(0, 4) for j in range(n)]
        add = [x if len(want[p]) + x <= M * R else 0 for x, p in zip(add, par)]
        vals = torch.randn(L, 24, D, device=DEV)
        parent.copy_(ints(par))
        n_new.copy_(ints(add))
        rows.copy_(vals)
        graphs[i & 1].replay()
        assert dsa.get_status() == 0
        f = oc.fork(par, *state, R, M)
        e = oc.extend(add, *f[:3], R, M, 24)
        state = e[:3]
        b = 1 - (i & 1)
        assert [t[b].tolist(), ln[b].tolist(), rf[b].tolist(), slots.tolist()] == list(e)
        want = [list(want[p]) for p in par]
        at = 0
        for j in range(n):
            for _ in range(add[j]):
                want[j].append(vals[:, at])
                at += 1
        for j in range(n):
            if want[j]:
                pos = torch.arange(len(want[j]), device=DEV)
                pg = t[b][j].long()[pos // R]
                assert torch.equal(pool[:, pg, pos % R], torch.stack(want[j], 1))


def test_refused_calls():
    dsa = lib()
    c = dsa.make_cache(n_seqs=2, n_pages=8, page_rows=4, max_pages=3)
    t, l, r = ints([[0] * 3] * 2), ints([0, 0]), ints([0] * 8)
    k, cp = ints([0]), ints([[0] * 3] * 5)
    with pytest.raises(dsa.DSAError) as e:  # the new table may not be the old one
        dsa.cache_fork(c, l.clone(), t, l, r, t, l.clone(), r.clone(), cp, k)
    assert e.value.code == dsa.DSA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        dsa.cache_fork(c, l.clone(), t[:1], l, r, t.clone(), l.clone(), r.clone(), cp, k)
    with pytest.raises(TypeError):
        dsa.cache_fork(c, l.clone().long(), t, l, r, t.clone(), l.clone(), r.clone(), cp, k)
    with pytest.raises(ValueError):
        dsa.cache_fork(c, l.cpu(), t, l, r, t.clone(), l.clone(), r.clone(), cp, k)
    pool = torch.zeros(8, 4, 16, device=DEV)
    with pytest.raises(ValueError):
        dsa.cache_copy_pages(c, pool[:, :, ::2], cp, k)
    with pytest.raises(ValueError):
        dsa.cache_copy_pages(c, pool[:7], cp, k)
    with pytest.raises(ValueError):
        dsa.cache_write(c, pool, torch.zeros(3, 16, device=DEV), ints([0, 1, 2, 3]))
    with pytest.raises(ValueError):
        dsa.cache_write(c, pool, torch.zeros(3, 16, device=DEV).half(), ints([0, 1, 2]))
    bad = dsa.dsa_pool(pool.data_ptr(), 2, 64, 256, 64)  # layers run into pages
    assert dsa.lib.dsa_cache_copy_pages(ctypes.byref(c), ctypes.byref(bad), cp.data_ptr(), k.data_ptr(), 1,
                                        None) == dsa.DSA_ERR_INVALID_ARG


@pytest.mark.parametrize("n", [3063, 3064, 3068, 3071, 4083, 4084, 4095, 4096, 8192])
def test_any_number_of_sequences(n):
    # the plans keep some numbers of each sequence in shared memory: below, around and above the 48 KB that
    # a kernel has without asking for more (fork 16, extend 12 bytes per sequence, each with some 150 fixed)
    rng = random.Random(n)
    R, P, M = 2, 2 * n, 2
    d = Device(lib(), n, R, P, M)
    table, lens, refs = random_state(rng, n, R, n, M)
    refs += [0] * (P - len(refs))
    n_new = [rng.randint(0, min(2, M * R - x)) for x in lens]
    got, st = d.extend(n_new, table, lens, refs, sum(n_new) + 5)
    assert st == 0 and got == list(oc.extend(n_new, table, lens, refs, R, M, sum(n_new) + 5))
    parent = [i if rng.random() < 0.9 else rng.randrange(n) for i in range(n)]
    got, st = d.fork(parent, table, lens, refs)
    assert st == 0 and got == list(oc.fork(parent, table, lens, refs, R, M))
    got, st = d.compact(table, lens, refs)
    assert st == 0 and got == list(oc.compact(table, lens, refs, R, M))


def test_a_launch_that_fails_leaves_nothing_behind():
    # a call on the legacy stream while another stream is captured is refused by the runtime; the
    # library's next call, of any kind, is not taken for the one that failed
    dsa = lib()
    rt = ctypes.CDLL("libcudart.so.13")
    d = Device(dsa, 2, 4, 8, 3)
    t, ln, rf = ints([[1, -1, -1], [2, -1, -1]]), ints([3, 4]), ints([0, 1, 1, 0, 0, 0, 0, 0])
    o = [torch.empty_like(t), torch.empty_like(ln), torch.empty_like(rf), ints([[0] * 3] * 2), ints([0])]
    S = 40000                                      # (longer rows than the selection sets attributes for)
    par, x = ints([0, 1]), torch.randn(4, S, device=DEV)
    idx = torch.empty(4, 8, dtype=torch.int32, device=DEV)
    p = dsa.make_params(B=1, S_q=4, S_k=S, H=1, d_qk=8, d_v=8, H_I=1, d_I=8, topk=8, scale=1.0, dtype="fp32",
                        q_row_offset=S - 4)
    dsa.cache_fork(d.c, par, t, ln, rf, *o)
    dsa.topk(p, x, 0, 4, idx)
    torch.cuda.synchronize()
    side, legacy, graph = ctypes.c_void_p(), torch.cuda.default_stream(), ctypes.c_void_p()
    assert legacy.cuda_stream == 0 and rt.cudaStreamCreate(ctypes.byref(side)) == 0
    assert rt.cudaStreamBeginCapture(side, 0) == 0
    try:
        with pytest.raises(dsa.DSAError) as e:
            dsa.cache_fork(d.c, par, t, ln, rf, *o, stream=legacy)
    finally:
        rt.cudaStreamEndCapture(side, ctypes.byref(graph))
        rt.cudaStreamDestroy(side)
        rt.cudaGetLastError()
    assert e.value.code == dsa.DSA_ERR_CUDA
    dsa.topk(p, x, 0, 4, idx)
    dsa.cache_fork(d.c, par, t, ln, rf, *o)
    torch.cuda.synchronize()
    assert dsa.get_status() == 0
    assert torch.equal(idx[3].sort().values, x[3].topk(8).indices.int().sort().values)


# more steps than one CTA takes on, more pages than one CTA takes on, both
@pytest.mark.parametrize("n,R,P,M", [(64, 4, 4000, 300), (9, 16, 20011, 40), (70, 3, 24000, 290)])
def test_a_cluster_that_cannot_carry_a_call_out_changes_nothing(n, R, P, M):
    rng = random.Random(P)
    d = Device(lib(), n, R, P, M)
    ids = rng.sample(range(P), P // 2)
    table, lens, refs = [], [], [0] * P
    for i in range(n):
        most = min(M, P // 2 // n)
        lens.append(rng.randint(most // 2, most - 2) * R + 1)  # a partial last page each
        row = [ids.pop() for _ in range(oc.pages_of(lens[i], R))]
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (M - len(row)))
    E, few = d.dsa.DSA_ERR_INDEX, d.dsa.DSA_ERR_PAGES
    same, grow = list(range(n)), [1] * n
    f = lambda parent=same, t=table, ln=lens, rf=refs: (d.fork(parent, t, ln, rf), ([t, ln, rf, []]))
    e = lambda n_new=grow, t=table, ln=lens, rf=refs: (d.extend(n_new, t, ln, rf, n + 3), [t, ln, rf, [-1] * (n + 3)])
    c = lambda t=table, ln=lens, rf=refs: (d.compact(t, ln, rf), [t, rf, [p if r > 0 else -1 for p, r in enumerate(rf)], []])

    def put(x, i, v):
        x = list(x)
        x[i] = v
        return x

    def check(result, code):
        (got, st), want = result
        assert st == code and got == want

    for i in (0, n // 2, n - 1):
        last = oc.pages_of(lens[i], R) - 1
        for page in (-1, P, 2 ** 31 - 1, -2 ** 31):
            for j in (0, last):
                bad = put(table, i, put(table[i], j, page))
                check(f(t=bad), E)
                check(c(t=bad), E)
            check(e(t=bad), E)                     # (the last page, into which the row goes)
        for ln in (-1, M * R + 1, 2 ** 31 - 1, -2 ** 31):
            check(f(ln=put(lens, i, ln)), E)
            check(e(ln=put(lens, i, ln)), E)
            check(c(ln=put(lens, i, ln)), E)
        for parent in (-2, n, 2 ** 31 - 1):
            check(f(parent=put(same, i, parent)), E)
        for a in (-1, M * R, n + 4):
            check(e(n_new=put(grow, i, a)), E)
        check(f(parent=put(same, i, -1), rf=put(refs, table[i][last], 0)), E)  # a count below the uses given up
        check(c(rf=put(refs, table[i][0], 0)), E)
        check(e(rf=put(refs, table[i][last], 2)), E)           # rows into a shared page
    for p in (0, P // 2, P - 1):
        if refs[p] == 0:
            for call in (f, e, c):
                check(call(rf=put(refs, p, -1)), E)
    # too few free pages: k of them, and one more needed (first of each request's children keeps its own)
    for k in (0, 3):
        free = [p for p, r in enumerate(refs) if r == 0]
        held = list(refs)
        for p in free[k:]:
            held[p] = 1
        n_new = [R if i <= k else 0 for i in same]             # a page each
        assert oc.extend(n_new, table, lens, held, R, M, n * R) is None
        got, st = d.extend(n_new, table, lens, held, n * R)
        assert st == few and got == [table, lens, held, [-1] * (n * R)]
        need = [0] * (k + 2) + same[k + 2:]        # k + 1 further children of sequence 0
        for i in range(1, k + 2):                  # their old pages would fall free: someone holds them
            for p in table[i][:oc.pages_of(lens[i], R)]:
                held[p] += 1
        assert oc.fork(need, table, lens, held, R, M) is None
        check(f(parent=need, rf=held), few)
