"""The run arithmetic of the cache pass (csrc/cache_attn.cu: Runs, Walk and parts_of, replayed
here in the same integer steps): every live tile is handed out once, segments have distinct
slots inside the workspace, and the join looks for exactly the segments that are written."""
import random

import pytest

TILE, SEGMENT = 64, 5


def tiles_of(n):
    return (n + TILE - 1) // TILE


def cost(t):
    return t + SEGMENT if t > 0 else 0


class Runs:
    def __init__(self, total, workers):
        self.n = min(total, workers)
        self.len = total // self.n if self.n else 0
        self.longer = total - self.n * self.len

    def start(self, w):
        return w * self.len + min(w, self.longer)

    def worker(self, x):
        split = self.longer * (self.len + 1)
        return x // (self.len + 1) if x < split else self.longer + (x - split) // self.len


def walk(lens, heads, runs, worker):
    """(plane, first tile, tiles) of a worker's segments, by the kernel's steps."""
    if worker >= runs.n:
        return
    at = runs.start(worker)
    left = runs.start(worker + 1) - at
    for b, n in enumerate(lens):
        own = cost(tiles_of(n)) * heads
        if at < own:
            break
        at -= own
    tiles = tiles_of(lens[b])
    kvh, t0 = at // cost(tiles), at % cost(tiles)

    def advance():
        nonlocal left, t0, kvh, b, tiles
        left -= cost(tiles) - t0
        t0 = 0
        if left <= 0:
            return
        kvh += 1
        if kvh < heads:
            return
        kvh, b = 0, b + 1
        while b < len(lens) and lens[b] == 0:
            b += 1
        if b == len(lens):
            left = 0
        else:
            tiles = tiles_of(lens[b])

    if t0 >= tiles:
        advance()
    while left > 0:
        yield b * heads + kvh, t0, min(left, tiles - t0)
        advance()


@pytest.mark.parametrize("seed", range(200))
def test_runs_cover_every_tile_once_and_the_join_finds_them(seed):
    rng = random.Random(seed)
    heads, workers = rng.choice([1, 2, 3, 8, 12]), rng.choice([148, 74, 5, 1])
    lens = [rng.choice([0, 1, 63, 64, 65, rng.randint(0, 300), rng.randint(0, 9000)]) for _ in range(rng.randint(1, 70))]
    runs = Runs(sum(cost(tiles_of(n)) for n in lens) * heads, workers)
    seen, slots = {}, {}
    for w in range(workers):
        for plane, t0, count in walk(lens, heads, runs, w):
            assert count > 0
            assert plane + w not in slots and plane + w < len(lens) * heads + workers
            slots[plane + w] = plane
            for t in range(t0, t0 + count):
                assert (plane, t) not in seen
                seen[plane, t] = w
    assert set(seen) == {(b * heads + h, t) for b, n in enumerate(lens) for h in range(heads) for t in range(tiles_of(n))}
    before = 0
    for b, n in enumerate(lens):
        t = tiles_of(n)
        for h in range(heads if t else 0):
            s0 = before * heads + h * cost(t)
            w0, w1 = runs.worker(s0), runs.worker(s0 + t - 1)
            plane = b * heads + h
            assert [plane + w for w in range(w0, w1 + 1)] == sorted(s for s, q in slots.items() if q == plane)
        before += cost(t)


@pytest.mark.parametrize("seed", range(100))
def test_a_prefix_as_the_last_sequence_has_slots_of_its_own(seed):
    # its segments are numbered head + worker in a buffer of their own, which holds
    # heads + workers of them, and the join finds them from the list's end
    rng = random.Random(1000 + seed)
    heads, workers = rng.choice([1, 2, 3, 8, 12]), 148
    lens = [rng.choice([0, 1, 64, 65, rng.randint(0, 3000)]) for _ in range(rng.randint(1, 32))]
    prefix = rng.choice([1, 64, 65, rng.randint(1, 500), rng.randint(1, 9000)])
    total = (sum(cost(tiles_of(n)) for n in lens) + cost(tiles_of(prefix))) * heads
    runs, slots = Runs(total, workers), {}
    for w in range(workers):
        for plane, t0, count in walk(lens + [prefix], heads, runs, w):
            kvh = plane - len(lens) * heads
            if kvh >= 0:
                assert kvh + w not in slots and kvh + w < heads + workers
                slots[kvh + w] = kvh
            else:
                assert plane + w < len(lens) * heads + workers       # the caches' slots stay inside theirs
    t = tiles_of(prefix)
    for h in range(heads):
        s0 = total - (heads - h) * cost(t)
        w0, w1 = runs.worker(s0), runs.worker(s0 + t - 1)
        assert [h + w for w in range(w0, w1 + 1)] == sorted(s for s, q in slots.items() if q == h)
