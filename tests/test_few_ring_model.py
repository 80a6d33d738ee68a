"""The ring of weight stages of moe_layer_few's 4-bit down pass as a model on the
CPU: which waits let a consumer team read a stage that has not landed.

Copies land in any order.  A wait by parity for a barrier's phase n passes when n
phases mod 2 tell it so: it takes phase n - 2's completion for phase n's while phase
n - 1 is under way.  Both teams meet at the end of a strip that they share; a solo
strip (of at most SHORT stages) is one team's alone, the teams taking such strips in
turn.  `ordered`: where a slot's last fill was the other team's, a team first waits
for it to be emptied: for the last such stage of a solo strip before the strip, and
before every stage of routed strips that follow solo ones of the shared expert."""
import os
import random
import re

import pytest

import mixture_experts_layer_gating_gb300 as moe

SHORT = 3  # stages of a solo strip, at most


class Misread(Exception):
    pass


class Stuck(Exception):
    pass


class Ring:
    """strips: the stages of every strip of a CTA's run (the first and the last may be
    parts); solo(c): whether a strip of that length in full is one team's."""

    def __init__(self, slots, strips, full_len, ordered):
        self.n = slots
        self.full = [0] * slots   # phases completed
        self.empty = [0] * slots
        self.landed = [set(), set()]  # stages whose copy, whose token rows are there
        self.flight = []
        # a team's programme: waits for a stage's slot to be emptied, stages, and the
        # meetings with the other team
        self.todo = [[], []]
        q, turn = 0, 0
        shared = full_len[0]  # strips of this length, at the run's start, are the shared expert's
        routed = next((i for i, c in enumerate(full_len) if c != shared), len(full_len))
        for i, (c, whole) in enumerate(zip(strips, full_len)):
            every = ordered and shared <= SHORT and i >= routed
            first = whole - c if i == 0 else 0  # the run begins inside a strip
            alone = whole <= SHORT
            if alone and ordered and not every:
                far = [j for j in range(first, first + c) if -(-(slots - j) // whole) % 2]
                if far:
                    self.todo[turn].append(("emptied", q + far[-1] - first))
            for t in (0, 1):
                for at in range(q, q + c) if alone and t == turn else [] if alone else range(q + t, q + c, 2):
                    if every:
                        self.todo[t].append(("emptied", at))
                    self.todo[t].append(at)
                if not alone:
                    self.todo[t].append(("meet", i))
            turn ^= alone
            q += c
        self.total = q
        self.issued = 0
        self.fed = [0, 1]  # the next stage of each feeder

    def _emptied(self, q):  # a wait by parity: the slot is free for stage q
        s, n = q % self.n, q // self.n
        return (self.empty[s] ^ n) & 1 == 0

    def _complete(self, q):
        if q in self.landed[0] and q in self.landed[1]:
            assert self.full[q % self.n] == q // self.n
            self.full[q % self.n] += 1

    def moves(self):
        out = []
        if self.issued < self.total and self._emptied(self.issued):
            out.append(("issue", self.issued))
        for f in (0, 1):
            if self.fed[f] < self.total and self._emptied(self.fed[f]):
                out.append(("feed", self.fed[f]))
        out += [("land", q) for q in self.flight]
        for t in (0, 1):
            if not self.todo[t]:
                continue
            q = self.todo[t][0]
            if isinstance(q, tuple) and q[0] == "emptied":
                if self._emptied(q[1]):
                    out.append(("go on", t))
                continue
            if isinstance(q, tuple):
                if self.todo[1 - t] and self.todo[1 - t][0] == q and t == 0:
                    out.append(("meet", q))
                continue
            s, n = q % self.n, q // self.n
            if (self.full[s] ^ n) & 1:
                out.append(("take", t))
        return out

    def do(self, move):
        what, q = move
        if what == "issue":
            self.flight.append(q)
            self.issued += 1
        elif what == "feed":
            self.fed[q & 1] += 2
            self.landed[1].add(q)
            self._complete(q)
        elif what == "land":
            self.flight.remove(q)
            self.landed[0].add(q)
            self._complete(q)
        elif what == "go on":
            at = self.todo[q].pop(0)[1]
            if self.empty[at % self.n] != at // self.n:
                raise Misread(f"team {q} takes stage {at - 2 * self.n} for the one before {at}")
        elif what == "meet":
            for t in (0, 1):
                self.todo[t].pop(0)
        else:
            at = self.todo[q].pop(0)
            if self.full[at % self.n] != at // self.n + 1:
                raise Misread(f"team {q} takes stage {at} before it has landed")
            assert self.empty[at % self.n] == at // self.n
            self.empty[at % self.n] += 1

    def run(self, late, rng):
        """Every move but those of `late` (stages whose copies come last) as it comes."""
        while True:
            moves = self.moves()
            if not moves:
                if any(self.todo):
                    raise Stuck
                return
            early = [m for m in moves if m[0] != "land" or m[1] not in late]
            self.do(rng.choice(early or moves))


# slots of the ring (8: up to eight tokens, 6: more), then the strips of a run and their full lengths
RUNS = [
    (8, [3] * 12, [3] * 12),
    (8, [1] + [3] * 8 + [2], [3] * 10),
    (6, [2] * 14, [2] * 14),
    (6, [1] * 20, [1] * 20),
    (6, [3] * 10, [3] * 10),
    (8, [2] + [3] * 11, [3] * 12),
    (8, [1] * 20, [1] * 20),
    (8, [1] + [2] * 14, [2] * 15),
    (6, [1] + [2] * 12 + [1], [2] * 14),
    (8, [9, 9] + [3] * 9, [9, 9] + [3] * 9),              # the shared expert's long strips first
    (6, [4, 9] + [2] * 9, [9, 9] + [2] * 9),
    (6, [2] * 5 + [6, 6, 6, 5], [2] * 5 + [6, 6, 6, 6]),  # its solo strips first
    (8, [3] * 3 + [4, 4, 4, 4, 1], [3] * 3 + [4] * 5),
    (8, [1, 3, 3] + [2] * 9, [3] * 3 + [2] * 9),          # both solo, of two lengths
    (6, [2] * 4 + [3] * 9, [2] * 4 + [3] * 9),
    (8, [1] * 7 + [3] * 8, [1] * 7 + [3] * 8),
    (6, [3] * 5 + [1] * 9, [3] * 5 + [1] * 9),
    (6, [5, 5, 5, 5, 4], [5] * 5),                        # no solo strips
    (8, [24, 31], [31, 31]),
]


def test_the_model_has_the_kernel_s_short_strips():
    src = os.path.join(os.path.dirname(moe.__file__), "csrc", "few_layer.cuh")
    with open(src) as f:
        assert int(re.search(r"constexpr int kFewShort = (\d+);", f.read()).group(1)) == SHORT


def _schedules(slots, strips, full_len, ordered):
    total = sum(strips)
    for late in [()] + [(a, b) for a in range(total) for b in {a, a + 1, (a + slots // 2) % total}]:
        for seed in range(3):
            yield Ring(slots, strips, full_len, ordered), set(late), random.Random(f"{late}{seed}")


@pytest.mark.parametrize("slots,strips,full_len", RUNS, ids=lambda v: str(v) if isinstance(v, int) else None)
def test_no_stage_is_read_before_it_landed(slots, strips, full_len):
    for ring, late, rng in _schedules(slots, strips, full_len, ordered=True):
        ring.run(late, rng)
        assert ring.issued == ring.total and sum(ring.empty) == ring.total


# (where the slots hold a whole number of pairs of strips, each stays with one team)
@pytest.mark.parametrize("slots,strips,full_len",
                         [r for r in RUNS if min(r[2]) <= SHORT and (len(set(r[2])) > 1 or r[0] % (2 * r[2][0]))],
                         ids=lambda v: str(v) if isinstance(v, int) else None)
def test_solo_strips_need_the_order(slots, strips, full_len):
    """Without the second wait some order of the copies is misread."""
    def misread():
        for ring, late, rng in _schedules(slots, strips, full_len, ordered=False):
            try:
                ring.run(late, rng)
            except (Misread, AssertionError, Stuck):
                return True
        return False

    assert misread()
