"""The order between the joins and the record slots of the tensor-core attention kernel (csrc/pa_attend_tc.cuh).

With at most one row tile per segment the two streams of a CTA take a segment's position tiles in turn, each leaves its part
of a whole segment in a record, and the stream that arrives last joins them.  The records of whole segments have two slots
by turns.  The model here holds the kernel's events (loads, products, weights, records, arrivals, joins) of one CTA, or of a
pair, with an edge for each program order and each barrier.  A slot may be written again only by an event that comes after
the join of the records in it, whichever stream joins.
"""

import itertools
import os
import random
import re

import pytest

TC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_144_gb300", "csrc",
                  "pa_attend_tc.cuh")


def slot_wait_in_source():
    """Whether the kernel waits for a slot's last join before it writes the slot, and says when a join is done."""
    with open(TC) as f:
        text = f.read()
    wait = re.search(r"if \(f\.whole\) \{[^\n]*\n[^\n]*wait\(Tr::JD \+ slot,", text)
    record = re.search(r"record_at<D>\(p, blockIdx\.x, slot_kind, e\)", text)
    join = re.search(r"join_rows<KVT, D, CG>\(p, f", text)
    done = re.search(r"mbar_arrive\(bar\(Tr::JD \+ slot\)\)", text)
    return bool(wait and record and join and done and wait.start() < record.start() < join.start() < done.start())


class Model:
    """Events of whole fragments of `tiles` position tiles each, in rings of `stages`, on `ranks` CTAs of a group."""

    def __init__(self, tiles, stages, ranks, joiners, slot_wait):
        self.after = {}                                   # event -> events that come after it
        self.tiles = tiles
        order = self._order
        starts = list(itertools.accumulate([0] + tiles))
        parity, frags = 0, []                             # per fragment: tile counts of stream 0 and 1
        for k, n in enumerate(tiles):
            own = [[], []]
            for i in range(n):
                own[(i & 1) ^ parity].append(starts[k] + i)
            parity ^= n & 1
            frags.append(own)
        stream_of = {c: t for own in frags for t in (0, 1) for c in own[t]}
        total = starts[-1]
        for r in range(ranks):                            # producers, one warp for K, one for queries and V
            last = None
            for c in range(total):
                if last:
                    order(last, ("K", r, c))
                last = ("K", r, c)
                if c >= stages:
                    order(("QK", c - stages, 1), last)
            last, used = None, [None, None]
            for k, own in enumerate(frags):
                first = stream_of[starts[k]]
                for t in (first, first ^ 1):
                    if not own[t]:
                        continue
                    load = ("Q", r, k, t)
                    if last:
                        order(last, load)
                    if used[t]:
                        order(used[t], load)
                    used[t], last = ("QK", own[t][-1], 1), load
                for c in range(starts[k], starts[k + 1]):
                    if last:
                        order(last, ("V", r, c))
                    last = ("V", r, c)
                    if c >= stages:
                        order(("PV", c - stages, 1), last)
        for t in (0, 1):                                  # issuers (of the group's first CTA), one warp per stream
            last = None

            def issue(event):
                nonlocal last
                if last:
                    order(last, event)
                last = event

            for k, own in enumerate(frags):
                mine = own[t]
                if not mine:
                    continue

                def scores(c, half):
                    issue(("QK", c, half))
                    for r in range(ranks):
                        order(("K", r, c), last)
                        order(("Q", r, k, t), last)

                scores(mine[0], 0)
                scores(mine[0], 1)
                for i, c in enumerate(mine):
                    for half in (0, 1):
                        issue(("PV", c, half))
                        for r in range(ranks):
                            order(("V", r, c), last)
                            order(("P", r, c, half), last)
                        if i + 1 < len(mine):
                            scores(mine[i + 1], half)
        self.reuse = []                                   # (join of a slot's use, record of its next use)
        for r in range(ranks):                            # softmax warps, one program order per stream
            uses = [None, None]
            lasts = [None, None]
            for k, own in enumerate(frags):
                for t in (0, 1):
                    for c in own[t]:
                        for half in (0, 1):
                            e = ("P", r, c, half)
                            order(("QK", c, half), e)
                            if lasts[t]:
                                order(lasts[t], e)
                            lasts[t] = e
                if not (own[0] and own[1]):               # a single tile is written out without a record
                    for t in (0, 1):
                        if own[t]:
                            order(("PV", own[t][-1], 1), ("out", r, k))
                            order(lasts[t], ("out", r, k))
                            lasts[t] = ("out", r, k)
                    continue
                slot = k & 1
                for t in (0, 1):
                    e = ("record", r, k, t)
                    order(("PV", own[t][-1], 1), e)
                    order(lasts[t], e)
                    lasts[t] = e
                    if uses[slot] is not None:
                        self.reuse.append((("join", r, uses[slot]), e))
                        if slot_wait:
                            order(("join", r, uses[slot]), e)
                j = joiners[r][k]
                order(("record", r, k, j ^ 1), ("join", r, k))   # the joining stream arrived last
                order(lasts[j], ("join", r, k))
                lasts[j] = ("join", r, k)
                uses[slot] = k

    def _order(self, a, b):
        self.after.setdefault(a, set()).add(b)
        self.after.setdefault(b, set())

    def reachable(self, a):
        seen, todo = set(), [a]
        while todo:
            for b in self.after[todo.pop()]:
                if b not in seen:
                    seen.add(b)
                    todo.append(b)
        return seen

    def acyclic(self):
        into = {a: 0 for a in self.after}
        for bs in self.after.values():
            for b in bs:
                into[b] += 1
        ready, done = [a for a, n in into.items() if n == 0], 0
        while ready:
            done += 1
            for b in self.after[ready.pop()]:
                into[b] -= 1
                if into[b] == 0:
                    ready.append(b)
        return done == len(into)

    def overwritten(self):
        """(join, record) pairs without an order between them."""
        reach = {}
        return [(j, w) for j, w in self.reuse if w not in reach.setdefault(j, self.reachable(j))]


def _joiners(rng, ranks, n):
    return [[rng.randrange(2) for _ in range(n)] for _ in range(ranks)]


BATCHES = [[n] * 7 for n in range(1, 9)] + [[2, 1, 2, 1, 2, 1, 2], [3, 2, 2, 3, 2, 2, 4], [2, 2, 1, 1, 3, 2, 2, 8, 2, 2]]


@pytest.mark.parametrize("stages", [2, 3, 4])
@pytest.mark.parametrize("ranks", [1, 2])
def test_a_record_is_joined_before_its_slot_is_written_again(stages, ranks):
    slot_wait = slot_wait_in_source()
    rng = random.Random(stages * 10 + ranks)
    batches = BATCHES + [[rng.randint(1, 5) for _ in range(10)] for _ in range(12)]
    for tiles in batches:
        for joiners in ([[0] * len(tiles)] * ranks, [[1] * len(tiles)] * ranks, _joiners(rng, ranks, len(tiles))):
            m = Model(tiles, stages, ranks, joiners, slot_wait)
            assert m.acyclic(), (tiles, joiners)                  # no wait of the kernel depends on itself
            assert not m.overwritten(), (tiles, joiners, m.overwritten()[0])


@pytest.mark.parametrize("stages", [2, 3, 4])
def test_the_model_finds_the_race_without_the_wait(stages):
    """Two tiles per segment: nothing but the wait keeps the stream that does not join from running ahead."""
    for tiles in ([2] * 5, [2, 1, 2, 1, 2]):
        assert Model(tiles, stages, 1, [[1] * 5], False).overwritten()
    assert not Model([8] * 5, stages, 1, [[1] * 5], False).overwritten()
