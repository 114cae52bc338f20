"""Executable model of the cache-attention kernel's mbarrier protocol (no GPU).

``cache_attn_kernel`` (csrc/cache_attn.cu) runs a worker's tiles, cut into segments (one per
plane), with two kinds of roles:

* the TMA producer (last warp): per segment the plane's Q rows into one of two slots, then K
  and V tiles into one ring (K of tile T at ring position 2T, V at 2T + 1);
* the consumer warps, in groups that take the tiles in turn (tile T goes to group T mod G).  A
  warp reads Q into registers and releases its slot, then for each of its group's tiles reads K
  (released after the scores), then V (released after the product).  At a segment's end the
  parts' (m, l, O) meet in shared memory: after a group barrier (the previous segment's have
  been read) each part that had a tile writes its slot, and after a second one every part reads
  those slots.

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
        self.QS = 1 if row_parts == 4 else 2
        for s in range(self.QS):
            self.barrier(f"q_full{s}", 1)
            self.barrier(f"q_empty{s}", self.warps)
            self.buffer(f"Q{s}")
        for s in range(2):
            self.barrier(f"group{s}", self.warps)
        for i in range(self.parts * row_parts):
            self.buffer(f"J{i}")
        self.done = []

    def roles(self):
        return [self.producer()] + [self.consumer(w) for w in range(self.warps)]

    def producer(self):
        u = 0
        for seg, n in enumerate(self.segments):
            qs = seg % self.QS
            if seg >= self.QS:
                yield from self.wait(f"q_empty{qs}", seg // self.QS - 1, "q_empty")
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
            qs, group0 = seg % self.QS, T % self.G
            yield from self.wait(f"q_full{qs}", seg // self.QS, "q_full")
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
            has_tile = [(i // (self.GW // self.WR) - group0) % self.G < n for i in range(self.parts)]
            yield from group_sync("read")
            if has_tile[part]:
                self.buf[f"J{part * self.WR + wr}"].write(("j", seg, part), f"w{w}")
                yield
            yield from group_sync("stored")
            for i in range(self.parts):
                if has_tile[i]:
                    self.buf[f"J{i * self.WR + wr}"].begin_read(("j", seg, i))
            yield
            for i in range(self.parts):
                if has_tile[i]:
                    self.buf[f"J{i * self.WR + wr}"].end_read()
            self.done.append((seg, w))

    def finished(self):
        if sorted(self.done) != [(seg, w) for seg in range(len(self.segments)) for w in range(self.warps)]:
            raise Hazard("a segment's parts were not joined once by every warp")


# (groups, warps per group, row parts, ring slots) as in the kernel: up to 8 rows; 16; 32; 64
FORMS = {"rows8": (5, 2, 1, 10), "rows8_d64": (5, 2, 1, 20), "rows16": (4, 2, 1, 8), "rows32": (4, 2, 2, 8), "rows64": (2, 4, 4, 8)}


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


@pytest.mark.parametrize("form", [(2, 4, 1, 5), (6, 2, 1, 10), (5, 2, 1, 12)])
def test_a_ring_shared_between_groups_is_caught(form):
    caught = 0
    for sched in range(200):
        try:
            _run(form, [9, 14, 3, 8], seed=sched)
        except Hazard:
            caught += 1
    assert caught > 0
