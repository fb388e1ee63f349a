"""The barriers of the tensor-core attention's key ring (tree_attn_tc.cu), as a model that
runs its roles under random schedules.

A barrier wait tests the parity of a phase, so it must not be possible that the
barrier completes two phases while a thread still stands before its wait: the
thread would then wait for a phase that depends on itself.  The model holds the
roles' order of waits and arrivals, counts whole phases, and takes every block as
one whose softmax waits for the last P V (to rescale O).
"""
import random

import pytest

STAGES = 3


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1


class Ring:
    def __init__(self, segments, release, seed, soft=3, fix=2):
        self.rng = random.Random(seed)
        self.segments, self.release, self.soft, self.fix = segments, release, soft, fix
        # blocks whose keys go past the fix warps
        self.plain = [self.rng.random() < 0.5 for _ in range(sum(segments) + len(segments))]
        self.full = [Barrier(1) for _ in range(STAGES)]
        self.empty = [Barrier(1 + fix) for _ in range(STAGES)]
        self.ready = [Barrier(fix) for _ in range(STAGES)]
        self.fixed = [Barrier(fix) for _ in range(STAGES)]
        self.s_full, self.s_free = Barrier(1), Barrier(soft)
        self.p_full = [Barrier(soft) for _ in range(2)]
        self.q_tm, self.q_free, self.done = ([Barrier(n) for _ in range(2)] for n in (fix, 1, 1))
        self.mma = [[], []]                         # commits of the two issuers that have not arrived yet

    # a role yields (barrier, phase) for a wait, None where another role may run
    def loads(self):
        slot = 0
        for blocks in self.segments:
            for j in range(1 + blocks):             # the query's slot, then the keys
                if slot >= STAGES:
                    yield self.empty[slot % STAGES], slot // STAGES - 1
                self.full[slot % STAGES].arrive()
                if j and self.plain[slot]:
                    yield None
                    for _ in range(self.fix):
                        self.ready[slot % STAGES].arrive()
                slot += 1

    def fixes(self):
        slot = 0
        for i, blocks in enumerate(self.segments):
            yield self.full[slot % STAGES], slot // STAGES
            if i:
                yield self.q_free[(i - 1) & 1], (i - 1) >> 1
            self.empty[slot % STAGES].arrive()
            self.fixed[slot % STAGES].arrive()
            self.q_tm[i & 1].arrive()
            slot += 1
            for _ in range(blocks):
                st = slot % STAGES
                yield self.full[st], slot // STAGES
                self.empty[st].arrive()
                self.fixed[st].arrive()
                if not self.plain[slot]:
                    self.ready[st].arrive()
                slot += 1

    def logits(self):
        slot = block = 0
        uses = [0] * STAGES
        for i, blocks in enumerate(self.segments):
            yield self.q_tm[i & 1], i >> 1
            query = self.empty[slot % STAGES]
            if self.release == "with the query":
                self.mma[0].append(query)
            slot += 1
            for j in range(blocks):
                st = slot % STAGES
                yield self.ready[st], uses[st]
                uses[st] += 1
                if block:
                    yield self.s_free, block - 1
                if j == 0 and self.release == "after s_free":
                    self.mma[0].append(query)
                if j >= 2:
                    yield self.empty[(slot - 2) % STAGES], (slot - 2) // STAGES
                self.mma[0].append(self.s_full)
                block += 1
                slot += 1
                yield None
            self.mma[0].append(self.q_free[i & 1])

    def values(self):
        slot = block = 0
        for i, blocks in enumerate(self.segments):
            slot += 1
            for _ in range(blocks):
                yield self.p_full[block & 1], block >> 1
                self.mma[1].append(self.empty[slot % STAGES])
                slot += 1
                block += 1
            self.mma[1].append(self.done[i & 1])

    def softmax(self):
        slot = block = 0
        for i, blocks in enumerate(self.segments):
            slot += 1
            for j in range(blocks):
                yield self.fixed[slot % STAGES], slot // STAGES
                yield self.s_full, block
                self.s_free.arrive()
                yield None
                if j:                               # the last P V, before O is rescaled
                    yield self.empty[(slot - 1) % STAGES], (slot - 1) // STAGES
                self.p_full[block & 1].arrive()
                slot += 1
                block += 1
            yield self.done[i & 1], i >> 1

    def tensor(self, k):                            # MMAs complete in order, at any time
        while True:
            if self.mma[k]:
                self.mma[k].pop(0).arrive()
            yield None

    def run(self):
        """'' or what went wrong."""
        rng = self.rng
        roles = {"loads": self.loads(), "logits": self.logits(), "values": self.values()}
        roles.update({f"fix {k}": self.fixes() for k in range(self.fix)})
        roles.update({f"softmax {k}": self.softmax() for k in range(self.soft)})
        engines = {"tensor 0": self.tensor(0), "tensor 1": self.tensor(1)}
        at = {name: None for name in (*roles, *engines)}
        slow = rng.choice(list(roles))              # one of them is late
        while roles:
            stuck = [n for n in roles if at[n] is not None and at[n][0].phase <= at[n][1]]
            if len(stuck) == len(roles) and not any(self.mma):
                return f"stopped: {stuck}"
            late = [n for n in roles if at[n] is not None and at[n][0].phase > at[n][1] + 1]
            if late:
                return f"two phases passed: {late}"
            ready = [n for n in roles if n not in stuck] + [e for k, e in enumerate(engines) if self.mma[k]]
            name = rng.choice(ready)
            if name == slow and len(ready) > 1 and rng.random() < 0.97:
                continue
            try:
                at[name] = next(engines[name] if name in engines else roles[name])
            except StopIteration:
                del roles[name]
        return ""


SEGMENTS = [[1], [1, 1, 1, 1], [2, 2, 2, 2, 2], [3, 3, 3], [7, 1, 2, 9, 4], [2, 5, 1, 1, 3, 2, 2]]


@pytest.mark.parametrize("segments", SEGMENTS)
def test_no_barrier_passes_two_phases_ahead_of_a_waiting_thread(segments):
    for seed in range(300):
        assert Ring(segments, "after s_free", seed).run() == ""


def test_the_model_sees_a_query_slot_released_too_early():
    # the slot two behind the last block but one holds the next tile's query: without the
    # softmax's word it can be free again while that block still waits for the P V before it
    found = [Ring([4, 4, 4], "with the query", seed).run() for seed in range(300)]
    assert any(f.startswith("two phases passed: ['softmax") for f in found)
