"""Executable model of the packed-attention kernel's mbarrier protocol (no GPU).

``packed_attn_kernel`` (csrc/packed.cu) runs a run of items per CTA with these roles:

* the K producer (warp 0): publishes each item in a ring of four, then loads its Q into one of
  two buffers and its K tiles into a 3-slot ring (the hardware's answer with the next item is
  this role's own business); after the last item it publishes an end mark;
* the V producer: V tiles into a ring of 2 or 3 slots; a tile past its sequence's end lands
  under ``v_tail`` and is completed by zeroing rows before ``v_full``;
* the Q K^T issuer: S(T) into TMEM buffer T mod 3 once P V of T - 3 is done;
* the P V issuer: O (+)= P(T) V; an item's first waits until the previous item's O is read;
* the softmax warps: per block read S and store P over it (a full block may be redone first,
  O may be rescaled); after an item's masked blocks they release the previous item's Q buffer,
  from which its O was stored asynchronously; at the end they read the next item, then O, and
  stage it in their rows of this item's Q buffer.

Built on ``tests.protocol_model`` (copies land in any order, each issuer's MMAs complete in
order; checks for deadlock, parity aliasing and buffer hazards).
"""
import random

import pytest

from tests.protocol_model import Hazard, ProtocolModel, random_decisions

NSB, KST, QST, RING = 3, 3, 2, 4
W = 2                                  # softmax warps modelled (8 in the kernel)


class PackedModel(ProtocolModel):
    issuers = ("qk", "pv")

    def __init__(self, items, vst, rng, omit=()):
        super().__init__(rng, omit)
        self.items, self.vst = items, vst              # (blocks, masked blocks, tail?)
        self.redo, self.rescale = random_decisions(rng, 0.2), random_decisions(rng, 0.2)
        for s in range(QST):
            self.barrier(f"q{s}", 1)
            self.barrier(f"q_empty{s}", 1 + W)
            for w in range(W):
                self.buffer(f"Q{s}w{w}")
        for s in range(KST):
            self.barrier(f"k_full{s}", 1)
            self.barrier(f"k_empty{s}", 1)
            self.buffer(f"K{s}")
        for s in range(vst):
            self.barrier(f"v_full{s}", 1)
            self.barrier(f"v_empty{s}", 1)
            self.buffer(f"V{s}")
        for b in range(NSB):
            self.barrier(f"s_full{b}", 1)
            self.barrier(f"p_full{b}", W)
            self.barrier(f"o_done{b}", 1)
            for w in range(W):
                self.buffer(f"S{b}w{w}")
        for name, count in (("o_free", W), ("v_tail", 1), ("final", 1), ("final_pv", 1)):
            self.barrier(name, count)
        for s in range(RING):
            self.barrier(f"item_full{s}", 1)
            self.barrier(f"item_empty{s}", W + 3)
            self.buffer(f"I{s}")
        for w in range(W):
            self.buffer(f"Ow{w}")
        self.stored = []

    def roles(self):
        return [self.k_producer(), self.v_producer(), self.qk(), self.pv()] + [self.softmax(w) for w in range(W)]

    def next_item(self, i):
        s = i % RING
        yield from self.wait(f"item_full{s}", i // RING, "item_full")
        self.buf[f"I{s}"].begin_read(("i", i))
        yield
        self.buf[f"I{s}"].end_read()
        self.bar[f"item_empty{s}"].arrive()

    def k_producer(self):
        T = nq = 0
        for i in range(len(self.items) + 1):
            s = i % RING
            if i >= RING:
                yield from self.wait(f"item_empty{s}", i // RING - 1, "item_empty")
            self.buf[f"I{s}"].write(("i", i), "k")
            self.bar[f"item_full{s}"].arrive()
            yield
            if i == len(self.items):
                return
            n = self.items[i][0]
            for t in range(n):
                if t == 0:
                    q = nq % QST
                    if nq >= QST:
                        yield from self.wait(f"q_empty{q}", nq // QST - 1, "q_empty")
                    # one copy, every warp's rows: the last lands the barrier
                    for w in range(W):
                        self.buf[f"Q{q}w{w}"].begin_write(("q", i), "tma")
                    self.loads.append((("Q", q), f"q{q}"))
                    nq += 1
                    yield
                k = T % KST
                if T >= KST:
                    yield from self.wait(f"k_empty{k}", T // KST - 1, "k_empty")
                self.tma(f"K{k}", ("k", T), f"k_full{k}")
                T += 1
                yield

    def fire(self, ev):
        kind, x = ev
        if kind == "load" and isinstance(self.loads[x][0], tuple):
            (_, q), barrier = self.loads.pop(x)
            for w in range(W):
                self.buf[f"Q{q}w{w}"].end_write()
            self.bar[barrier].arrive()
        else:
            super().fire(ev)

    def v_producer(self):
        T = tails = 0
        for i, (n, _, tail) in enumerate(self.items):
            yield from self.next_item(i)
            for t in range(n):
                s = T % self.vst
                if T >= self.vst:
                    yield from self.wait(f"v_empty{s}", T // self.vst - 1, "v_empty")
                if tail and t == 0:
                    self.tma(f"V{s}", ("raw", T), "v_tail")
                    yield
                    yield from self.wait("v_tail", tails, "v_tail")
                    tails += 1
                    self.buf[f"V{s}"].write(("v", T), "v")
                    self.bar[f"v_full{s}"].arrive()
                else:
                    self.tma(f"V{s}", ("v", T), f"v_full{s}")
                T += 1
                yield
        yield from self.next_item(len(self.items))

    def qk(self):
        T = nq = 0
        for i, (n, _, _) in enumerate(self.items):
            yield from self.next_item(i)
            if n == 0:
                continue
            q = nq % QST
            yield from self.wait(f"q{q}", nq // QST, "q_full")
            for _ in range(n):
                k, b = T % KST, T % NSB
                yield from self.wait(f"k_full{k}", T // KST, "k_full")
                if T >= NSB:
                    yield from self.wait(f"o_done{b}", T // NSB - 1, "s_reuse")
                self.issue_mma("qk", [(f"Q{q}w{w}", ("q", i)) for w in range(W)] + [(f"K{k}", ("k", T))],
                               [(f"S{b}w{w}", ("s", T), None) for w in range(W)])
                self.commit("qk", f"s_full{b}")
                self.commit("qk", f"k_empty{k}")
                T += 1
                yield
            self.commit("qk", f"q_empty{q}")
            nq += 1
        yield from self.next_item(len(self.items))
        self.commit("qk", "final")
        yield from self.wait("final", 0, "final")

    def pv(self):
        T = nq = 0
        for i, (n, _, _) in enumerate(self.items):
            yield from self.next_item(i)
            if n == 0:
                continue
            if nq > 0:
                yield from self.wait("o_free", nq - 1, "o_free")
            for t in range(n):
                s, b = T % self.vst, T % NSB
                yield from self.wait(f"p_full{b}", T // NSB, "p_full")
                yield from self.wait(f"v_full{s}", T // self.vst, "v_full")
                self.issue_mma("pv", [(f"S{b}w{w}", ("p", T)) for w in range(W)] + [(f"V{s}", ("v", T))],
                               [(f"Ow{w}", ("o", i, t), ("o", i, t - 1) if t else None) for w in range(W)])
                self.commit("pv", f"v_empty{s}")
                self.commit("pv", f"o_done{b}")
                T += 1
                yield
            nq += 1
        yield from self.next_item(len(self.items))
        self.commit("pv", "final_pv")
        yield from self.wait("final_pv", 0, "final")

    def softmax(self, w):
        T = nq = 0
        pending = False
        yield from self.next_item(0)
        for i, (n, masked, _) in enumerate(self.items):
            def release():
                nonlocal pending
                if pending:
                    self.buf[f"Q{(nq - 1) % QST}w{w}"].end_read()      # the copies have read it
                    self.bar[f"q_empty{(nq - 1) % QST}"].arrive()
                    pending = False
            for t in range(n):
                if t == masked:
                    release()
                b = T % NSB
                for _ in range(2 if t >= masked and t > 0 and self.redo(T, w) else 1):
                    yield from self.wait(f"s_full{b}", T // NSB, "s_full")
                    self.buf[f"S{b}w{w}"].begin_read(("s", T))
                    yield
                    self.buf[f"S{b}w{w}"].end_read()
                self.buf[f"S{b}w{w}"].write(("p", T), f"w{w}")
                yield
                if t >= 1 and self.rescale(T, w):
                    yield from self.wait(f"o_done{(T - 1) % NSB}", (T - 1) // NSB, "rescale")
                    self.buf[f"Ow{w}"].begin_write(("o", i, t - 1), f"w{w}", ("o", i, t - 1))
                    yield
                    self.buf[f"Ow{w}"].end_write()
                self.bar[f"p_full{b}"].arrive()
                T += 1
                yield
            release()
            yield from self.next_item(i + 1)
            if n:
                yield from self.wait(f"o_done{(T - 1) % NSB}", (T - 1) // NSB, "o_last")
                self.buf[f"Ow{w}"].begin_read(("o", i, n - 1))
                yield
                self.buf[f"Ow{w}"].end_read()
                self.bar["o_free"].arrive()
                q = f"Q{nq % QST}w{w}"
                self.buf[q].write(("out", i), f"w{w}")
                self.buf[q].begin_read(("out", i))
                nq += 1
                pending = True
                yield
            self.stored.append((i, w))
        if pending:
            self.buf[f"Q{(nq - 1) % QST}w{w}"].end_read()

    def finished(self):
        if sorted(self.stored) != [(i, w) for i in range(len(self.items)) for w in range(W)]:
            raise Hazard("an item was not stored once by every warp")


def _items(rng):
    out = []
    for _ in range(rng.randint(1, 7)):
        n = rng.choice([0, 1, 1, 2, 3, 4, 7])
        out.append((n, rng.randint(0, min(n, 2)), n > 0 and rng.random() < 0.5))
    return out


def _run(items, vst, seed, omit=()):
    PackedModel(items, vst, random.Random(seed), omit).run()


@pytest.mark.parametrize("vst", [2, 3])
def test_random_items_and_schedules(vst):
    for case in range(60):
        items = _items(random.Random(case))
        for sched in range(3):
            _run(items, vst, seed=100 * case + sched)


WAITS = ["item_full", "item_empty", "q_empty", "k_empty", "v_empty", "v_tail", "q_full", "k_full", "v_full", "s_reuse", "p_full",
         "s_full", "rescale", "o_last"]


@pytest.mark.parametrize("omit", WAITS)
def test_every_wait_is_needed(omit):
    caught = 0
    for sched in range(400):
        try:
            _run([(3, 1, True), (4, 0, False), (1, 1, True), (2, 1, False), (5, 1, True), (1, 1, False)] + 7 * [(0, 0, False)], 2,
                 seed=sched, omit=(omit,))
        except Hazard:
            caught += 1
            if caught >= 3:
                break
    assert caught > 0, f"no schedule needs the {omit} wait"


@pytest.mark.parametrize("omit", ["o_free", "final"])
def test_waits_implied_on_the_normal_path(omit):
    """o_free follows from p_full (a warp's next P follows its read of O); the issuers' drains
    from the softmax's waits.  Both stay: an explicit hand-off, and the abort path."""
    for sched in range(100):
        _run([(3, 1, True), (4, 0, False), (1, 1, True), (2, 1, False)], 2, seed=sched, omit=(omit,))
