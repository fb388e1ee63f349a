"""Paged-cache bookkeeping in plain Python: the definition the device calls are held to.

State: table (list of lists), lens, refs.  Each function returns the new state and
leaves its arguments alone; a call that cannot be carried out returns None.
"""
from __future__ import annotations


def pages_of(n, R):
    return -(-n // R)


def _held(table, lens, R, i):
    return table[i][:pages_of(lens[i], R)]


def _valid(table, lens, refs, R, max_pages):
    for i, n in enumerate(lens):
        if n < 0 or n > max_pages * R:
            return False
        if any(p < 0 or p >= len(refs) for p in _held(table, lens, R, i)):
            return False
    return all(r >= 0 for r in refs)


def fork(parent, table, lens, refs, R, max_pages):
    """(table, lens, refs, copies) after sequence i became a copy of old sequence parent[i]."""
    n = len(lens)
    if not _valid(table, lens, refs, R, max_pages) or any(p < -1 or p >= n for p in parent):
        return None
    refs = list(refs)
    for i in range(n):
        for p in _held(table, lens, R, i):
            refs[p] -= 1
    new_table, new_lens, needy, seen = [], [], [], set()
    for i, p in enumerate(parent):
        row = list(_held(table, lens, R, p)) if p >= 0 else []
        new_lens.append(lens[p] if p >= 0 else 0)
        if p >= 0 and p in seen and lens[p] % R:
            needy.append(i)
            row[-1] = -1
        seen.add(p)
        for x in row:
            if x >= 0:
                refs[x] += 1
        new_table.append(row)
    if any(r < 0 for r in refs):
        return None
    free = [p for p, r in enumerate(refs) if r == 0]
    if len(free) < len(needy):
        return None
    copies = []
    for i, page in zip(needy, free):
        src = table[parent[i]][pages_of(lens[parent[i]], R) - 1]
        copies.append((src, page, lens[parent[i]] % R))
        new_table[i][-1] = page
        refs[page] = 1
    return [r + [-1] * (max_pages - len(r)) for r in new_table], new_lens, refs, copies


def extend(n_new, table, lens, refs, R, max_pages, n_slots):
    """(table, lens, refs, slots) with room for n_new[i] more rows."""
    for i, (n, a) in enumerate(zip(lens, n_new)):
        if n < 0 or a < 0 or n + a > max_pages * R:
            return None
        if a and n % R:
            page = table[i][n // R]
            if page < 0 or page >= len(refs) or refs[page] != 1:
                return None
    if sum(n_new) > n_slots or any(r < 0 for r in refs):
        return None
    table, refs = [list(r) for r in table], list(refs)
    free = [p for p, r in enumerate(refs) if r == 0]
    slots = []
    for i, (n, a) in enumerate(zip(lens, n_new)):
        for j in range(pages_of(n, R), pages_of(n + a, R)):
            if not free:
                return None
            table[i][j] = free.pop(0)
            refs[table[i][j]] = 1
        slots += [table[i][x // R] * R + x % R for x in range(n, n + a)]
    return table, [n + a for n, a in zip(lens, n_new)], refs, slots + [-1] * (n_slots - len(slots))


def compact(table, lens, refs, R, max_pages):
    """(table, refs, map, copies) with the used pages at the lowest ids."""
    if not _valid(table, lens, refs, R, max_pages):
        return None
    if any(refs[p] == 0 for i in range(len(lens)) for p in _held(table, lens, R, i)):
        return None
    n_live = sum(r > 0 for r in refs)
    movers = [p for p, r in enumerate(refs) if r > 0 and p >= n_live]
    holes = [p for p, r in enumerate(refs) if r == 0 and p < n_live]
    new = {p: p for p, r in enumerate(refs) if r > 0}
    new.update(zip(movers, holes))
    refs_out = [0] * len(refs)
    for p, q in new.items():
        refs_out[q] = refs[p]
    rows = [[new[p] for p in _held(table, lens, R, i)] for i in range(len(lens))]
    return ([r + [-1] * (max_pages - len(r)) for r in rows], refs_out, [new.get(p, -1) for p in range(len(refs))],
            [(p, q, R) for p, q in zip(movers, holes)])
