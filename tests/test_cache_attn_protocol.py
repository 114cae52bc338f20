"""Executable model of the cache-attention kernel's mbarrier protocol (no GPU).

``cache_attn_kernel`` (csrc/cache_attn.cu) runs a worker's tiles, cut into segments (one per
plane), with two kinds of roles:

* the TMA producer (last warp): per segment the plane's Q rows into one of two slots, then K
  and V tiles into one ring (K of tile T at ring position 2T, V at 2T + 1);
* the consumer warps, in groups that take the tiles in turn (tile T goes to group T mod G).  A
  warp reads Q into registers and releases its slot, then for each of its group's tiles reads K
  (released after the scores), then V (released after the product).  At a segment's end the
  parts' (m, l, O) meet in a tree: of n parts the upper n / 2 write to a slot and, after a
  group barrier, are added by the lower ones; the upper part h + i uses slot i in the first
  round, later a part writes to the slot of its own number.

Built on ``tests.protocol_model`` (copies land in any order; checks for deadlock, parity
aliasing and buffer hazards).  A ring that does not hold a multiple of G tiles is caught: a
group's wait on a slot whose tile before, another group's, has not landed aliases.
"""
import random

import pytest

from tests.protocol_model import Hazard, ProtocolModel


class CacheModel(ProtocolModel):
    def __init__(self, segments, groups, group_warps, row_parts, slots, rng, omit=()):
        super().__init__(rng, omit)
        self.segments, self.G, self.GW, self.WR, self.slots = segments, groups, group_warps, row_parts, slots
        self.warps = groups * group_warps
        self.parts = groups * (group_warps // row_parts)
        for s in range(slots):
            self.barrier(f"full{s}", 1)
            self.barrier(f"empty{s}", group_warps)
            self.buffer(f"KV{s}")
        for s in range(2):
            self.barrier(f"q_full{s}", 1)
            self.barrier(f"q_empty{s}", self.warps)
            self.barrier(f"group{s}", self.warps)
            self.buffer(f"Q{s}")
        for i in range((self.parts + 1) // 2 * row_parts):
            self.buffer(f"J{i}")
        self.done = []

    def roles(self):
        return [self.producer()] + [self.consumer(w) for w in range(self.warps)]

    def producer(self):
        u = 0
        for seg, n in enumerate(self.segments):
            qs = seg & 1
            if seg >= 2:
                yield from self.wait(f"q_empty{qs}", (seg >> 1) - 1, "q_empty")
            self.tma(f"Q{qs}", ("q", seg), f"q_full{qs}")
            yield
            for _ in range(2 * n):
                s = u % self.slots
                if u >= self.slots:
                    yield from self.wait(f"empty{s}", u // self.slots - 1, "empty")
                self.tma(f"KV{s}", ("kv", u), f"full{s}")
                u += 1
                yield

    def consumer(self, w):
        group, wr = w // self.GW, (w % self.GW) % self.WR
        part = group * (self.GW // self.WR) + (w % self.GW) // self.WR
        T = seq = 0

        def group_sync(tag):
            nonlocal seq
            slot, phase = seq & 1, seq >> 1
            seq += 1
            self.bar[f"group{slot}"].arrive()
            yield from self.wait(f"group{slot}", phase, tag)

        for seg, n in enumerate(self.segments):
            qs = seg & 1
            yield from self.wait(f"q_full{qs}", seg >> 1, "q_full")
            self.buf[f"Q{qs}"].begin_read(("q", seg))
            yield
            self.buf[f"Q{qs}"].end_read()
            self.bar[f"q_empty{qs}"].arrive()
            for _ in range(n):
                if T % self.G == group:
                    for u in (2 * T, 2 * T + 1):
                        s = u % self.slots
                        yield from self.wait(f"full{s}", u // self.slots, "full")
                        self.buf[f"KV{s}"].begin_read(("kv", u))
                        yield
                        self.buf[f"KV{s}"].end_read()
                        self.bar[f"empty{s}"].arrive()
                T += 1
            total, first, m = {part}, True, self.parts
            while m > 1:
                h = (m + 1) // 2
                if h <= part < m:
                    slot = (part - h if first else part) * self.WR + wr
                    self.buf[f"J{slot}"].write(("j", seg, part, frozenset(total)), f"w{w}")
                    yield
                yield from group_sync("stored")
                if part < m - h:
                    slot = (part if first else part + h) * self.WR + wr
                    held = self.buf[f"J{slot}"].version
                    if held is None or held[:3] != ("j", seg, part + h) or total & held[3]:
                        raise Hazard(f"join of segment {seg}: part {part} reads {held}")
                    self.buf[f"J{slot}"].begin_read(held)
                    yield
                    self.buf[f"J{slot}"].end_read()
                    total |= held[3]
                first, m = False, h
            yield from group_sync("read")
            if part == 0:
                self.done.append((seg, wr, frozenset(total)))

    def finished(self):
        want = {(seg, wr, frozenset(range(self.parts))) for seg in range(len(self.segments)) for wr in range(self.WR)}
        if set(self.done) != want or len(self.done) != len(want):
            raise Hazard("a segment's parts were not joined once each")


# (groups, warps per group, row parts, ring slots) as in the kernel: up to 8 rows; 16; 32; 64
FORMS = {"rows8": (6, 2, 1, 12), "rows8_d64": (6, 2, 1, 24), "rows16": (4, 2, 1, 8), "rows32": (4, 2, 2, 8), "rows64": (2, 4, 4, 8)}


def _run(form, segments, seed, omit=()):
    CacheModel(segments, *form, random.Random(seed), omit).run()


@pytest.mark.parametrize("name", list(FORMS))
def test_random_segments_and_schedules(name):
    for case in range(25):
        rng = random.Random(case)
        segments = [rng.choice([1, 1, 2, 3, 5, 9, 14]) for _ in range(rng.randint(1, 4))]
        for sched in range(3):
            _run(FORMS[name], segments, seed=100 * case + sched)


@pytest.mark.parametrize("omit", ["q_full", "full", "empty", "stored", "q_empty", "read"])
def test_every_wait_is_needed(omit):
    caught = 0
    for sched in range(400):
        try:
            _run(FORMS["rows16"], [1, 2, 9, 1, 1, 6, 2], seed=sched, omit=(omit,))
        except Hazard:
            caught += 1
            if caught >= 3:
                break
    assert caught > 0, f"no schedule needs the {omit} wait"


@pytest.mark.parametrize("form", [(2, 4, 1, 5), (6, 2, 1, 10)])
def test_a_ring_shared_between_groups_is_caught(form):
    caught = 0
    for sched in range(200):
        try:
            _run(form, [9, 14, 3, 8], seed=sched)
        except Hazard:
            caught += 1
    assert caught > 0
