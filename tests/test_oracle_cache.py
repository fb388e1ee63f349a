"""The plain paged-cache bookkeeping: hand-worked steps, and what holds after any run of them."""
import random

from oracle import cache as oc


def test_hand_worked_fork_extend_compact():
    R = 4
    # sequence 0: 6 rows on pages 3, 1; sequence 1: 4 rows on page 3 (shared); sequence 2 empty
    table, lens = [[3, 1, -1], [3, -1, -1], [-1, -1, -1]], [6, 4, 0]
    refs = [0, 1, 0, 2, 0]
    t, l, r, copies = oc.fork([0, 0, 1], table, lens, refs, R, 3)
    # sequence 1 needs its own copy of the 2 rows on page 1: the lowest free page is 0
    assert (t, l) == ([[3, 1, -1], [3, 0, -1], [3, -1, -1]], [6, 6, 4])
    assert r == [1, 1, 0, 3, 0] and copies == [(1, 0, 2)]
    t, l, r, slots = oc.extend([3, 0, 1], t, l, r, R, 3, 6)
    assert t == [[3, 1, 2], [3, 0, -1], [3, 4, -1]] and l == [9, 6, 5]
    assert slots == [1 * 4 + 2, 1 * 4 + 3, 2 * 4 + 0, 4 * 4 + 0, -1, -1] and r == [1, 1, 1, 3, 1]
    t, l, r, copies = oc.fork([-1, 2, -1], t, l, r, R, 3)
    assert t == [[-1] * 3, [3, 4, -1], [-1] * 3] and r == [0, 0, 0, 1, 1] and copies == []
    t, r, m, copies = oc.compact(t, l, r, R, 3)
    assert t[1] == [0, 1, -1] and r == [1, 1, 0, 0, 0] and m == [-1, -1, -1, 0, 1]
    assert copies == [(3, 0, 4), (4, 1, 4)]


def test_refusals():
    assert oc.fork([1], [[0]], [2], [1], 4, 1) is None            # no such parent
    assert oc.fork([0], [[7]], [2], [1], 4, 1) is None            # no such page
    assert oc.fork([0, 0], [[0], [-1]], [2, 0], [1], 4, 1) is None  # no free page for the second child
    assert oc.extend([3], [[0]], [2], [1], 4, 1, 8) is None       # more rows than the table holds
    assert oc.extend([1], [[0]], [2], [2], 4, 1, 8) is None       # the last page is shared
    assert oc.extend([2], [[0, -1]], [2], [1], 4, 2, 1) is None   # more rows than slots
    assert oc.extend([3], [[0, -1]], [2], [1], 4, 2, 8) is None   # no free page


def test_contents_follow_every_step():
    # the rows of each sequence, kept apart as lists, always equal what the pages hold
    rng = random.Random(5)
    R, n, P, M = 3, 5, 60, 12
    table, lens, refs = [[-1] * M for _ in range(n)], [0] * n, [0] * P
    pool, want = [[None] * R for _ in range(P)], [[] for _ in range(n)]
    token = 0
    for step in range(200):
        what = rng.random()
        if what < 0.4:
            parent = [rng.choice([i, i, rng.randrange(n), -1]) for i in range(n)]
            got = oc.fork(parent, table, lens, refs, R, M)
            assert got is not None
            table, lens, refs, copies = got
            want = [list(want[p]) if p >= 0 else [] for p in parent]
        elif what < 0.85:
            a = [rng.randrange(0, 5) if lens[i] < M * R - 5 else 0 for i in range(n)]
            table, lens, refs, slots = oc.extend(a, table, lens, refs, R, M, 40)
            copies, k = [], 0
            for i in range(n):
                for _ in range(a[i]):
                    pool[slots[k] // R][slots[k] % R] = token
                    want[i].append(token)
                    token, k = token + 1, k + 1
        else:
            table, refs, _, copies = oc.compact(table, lens, refs, R, M)
            assert all(r > 0 for r in refs[:sum(r > 0 for r in refs)])
        for s, d, rows in copies:
            pool[d][:rows] = pool[s][:rows]
        held = [p for i in range(n) for p in table[i][:oc.pages_of(lens[i], R)]]
        assert refs == [held.count(p) for p in range(P)]
        for i in range(n):
            assert [pool[table[i][x // R]][x % R] for x in range(lens[i])] == want[i]
