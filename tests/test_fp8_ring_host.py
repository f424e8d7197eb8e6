"""The protocol between the warps of gdn_attn_paged_fp8's kernel, as a model with random scheduling (no GPU needed): a ring of
stages filled by feeding warps through copies that land at any time and taken by key groups, jobs in slots, and the turns in
which the key groups join.  Barriers are counted and waits tell two phases apart, as the hardware's do.  For every shape in the
kernel's source: no deadlock, no arrival too many, no tile, job or sum read before it is there or after it has been
overwritten, and no copy in flight at the end -- also where waits run out and warps give up, at any place.
"""
import math
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "serving_gdn_decode_gb300", "csrc", "attn_fp8.cu")


def shapes():
    """(WARPS, RW, FEED, STAGES, slots) of the kernel's variants, f32 and bf16: Pick8's arithmetic."""
    with open(SOURCE) as f:
        picks = [x.split(", ") for x in re.findall(r"f\(Pick8<T, ([^>]*)>\{\}\)", f.read())]
    assert len(picks) == 12 and all(len(x) in (8, 9) for x in picks)
    out = set()
    for size in (2, 4):
        def value(text):  # a number, a truth value, or either for f32 and for bf16
            both = re.fullmatch(r"f32 \? (\w+) : (\w+)", text)
            if both:
                return value(both[1] if size == 4 else both[2])
            return int(text) if text.isdigit() else {"true": True, "false": False, "f32": size == 4}[text]

        for pick in picks:
            d, nt, rw, warps, feed, kt, ctas, boxed, in_smem = [value(x) for x in pick] + [False] * (9 - len(pick))
            rows, tile, groups = nt * rw * 8, 16 * kt, 2 * kt if boxed else 16 * kt
            q_bytes = rows * (d * size + 16)
            slots = 4 if q_bytes <= 2400 else 3 if q_bytes <= 4800 else 2
            fragments = slots * rw * (d // 16 * nt * (2 if size == 4 else 1) * 256 if in_smem else 0)
            fixed = rw * (d // 16 * 4 + 4) * nt * 128 + slots * q_bytes + fragments
            fit = (228 * 1024 // ctas - 1024 - 1024 - 512 - 64 * warps * nt - 24 * 32 - fixed) // (2 * tile * d + 2 * groups * 4)
            turn = math.lcm(warps // rw, feed)
            out.add((warps, rw, feed, min(fit, 32) // turn * turn, slots))
    return sorted(out)


class Broken(Exception):
    pass


def need(ok, what):
    if not ok:
        raise Broken(what)


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        need(self.pending >= 1, "an arrival too many")
        self.pending -= 1
        if self.pending == 0:
            self.phase ^= 1
            self.pending = self.count

    def ended(self, parity):
        return self.phase != parity


class GaveUp(Exception):
    pass


class Cta:
    """One CTA's share.  `patience`: the chance that a wait which has not ended runs out at a look; `without`: parts of the
    protocol to leave out."""

    def __init__(self, shape, seed, patience=0.0, without=()):
        self.WARPS, self.RW, self.FEED, self.STAGES, self.SLOTS = shape
        self.KW = self.WARPS // self.RW
        self.r = random.Random(seed)
        self.patience, self.without, self.failed = patience, without, False
        self.items = [self.r.choice([0, 1, 1, 2, 3, 5, 17, 64]) for _ in range(self.r.randint(1, 30))]
        self.full = [Barrier(1) for _ in range(self.STAGES)]
        self.empty = [Barrier(self.RW) for _ in range(self.STAGES)]
        self.job_full = [Barrier(1) for _ in range(self.SLOTS)]
        self.job_empty = [Barrier(self.WARPS) for _ in range(self.SLOTS)]
        self.turns = [[Barrier(1) for _ in range(self.KW)] for _ in range(self.RW)]
        self.tiles, self.jobs, self.sums = [None] * self.STAGES, [None] * self.SLOTS, [None] * self.RW
        self.in_flight, self.put = [], set()

    def wait(self, barrier, parity, bounded=True):
        while not barrier.ended(parity):
            if bounded and (self.failed or self.r.random() < self.patience):
                if not barrier.ended(parity):  # looked at once more
                    self.failed = True
                    raise GaveUp
            yield

    def feeder(self, me):
        stage, phase, skip, slot, job_phase, filled, slots_filled = me, 1, me, 0, 1, False, False
        try:
            for item, n in enumerate(self.items + [None]):
                if me == self.FEED - 1:
                    yield from self.wait(self.job_empty[slot], job_phase)
                    self.in_flight.append((self.jobs, slot, item if n is not None else "none", self.job_full))
                    slot += 1
                    if slot == self.SLOTS:
                        slot, job_phase, slots_filled = 0, job_phase ^ 1, True
                if n is None:
                    break
                for tile in range(skip, n, self.FEED):
                    yield from self.wait(self.empty[stage], phase)
                    self.in_flight.append((self.tiles, stage, (item, tile), self.full))
                    yield
                    stage += self.FEED
                    if stage >= self.STAGES:
                        stage, phase, filled = stage - self.STAGES, phase ^ 1, True
                skip = (skip + self.FEED - n % self.FEED) % self.FEED
        except GaveUp:
            pass
        if "drain" in self.without:
            return
        for x in range(me, self.STAGES, self.FEED):
            if x < stage or filled:
                yield from self.wait(self.full[x], phase ^ 1 if x < stage else phase, bounded=False)
        if me == self.FEED - 1:
            for x in range(self.SLOTS):
                if x < slot or slots_filled:
                    yield from self.wait(self.job_full[x], job_phase ^ 1 if x < slot else job_phase, bounded=False)

    def taker(self, warp):
        group, rg = divmod(warp, self.RW)
        ahead = stage = group
        phase = slot = job_phase = turn_phase = 0
        turns = self.turns[rg]
        try:
            for item, n in enumerate(self.items + [None]):
                yield from self.wait(self.job_full[slot], job_phase)
                need(self.jobs[slot] == (item if n is not None else "none"), "a job that is not there")
                if n is None:
                    return
                while ahead < n:
                    yield from self.wait(self.full[stage], phase)
                    for _ in range(self.r.randint(0, 5)):
                        need(self.tiles[stage] == (item, ahead), "a tile that is not there")
                        yield
                    need(self.tiles[stage] == (item, ahead), "a tile that is not there")
                    self.empty[stage].arrive()
                    stage += self.KW
                    if stage >= self.STAGES:
                        stage, phase = stage - self.STAGES, phase ^ 1
                    ahead += self.KW
                ahead -= n
                turn = ahead
                if "last join" not in self.without:
                    yield from self.wait(turns[self.KW - 1], turn_phase ^ 1)
                if turn:
                    yield from self.wait(turns[turn - 1], turn_phase)
                    need(self.sums[rg] == (item, turn - 1), "sums that are not there")
                turn_phase ^= 1
                for _ in range(self.r.randint(0, 4)):
                    yield
                if turn == self.KW - 1:
                    self.put.add((item, rg))
                self.sums[rg] = (item, turn)
                turns[turn].arrive()
                need(self.jobs[slot] == item, "a job that is gone")
                self.job_empty[slot].arrive()
                slot += 1
                if slot == self.SLOTS:
                    slot, job_phase = 0, job_phase ^ 1
        except GaveUp:
            pass

    def run(self):
        warps = [self.feeder(i) for i in range(self.FEED)] + [self.taker(i) for i in range(self.WARPS)]
        idle = 0
        while warps:
            if self.in_flight and self.r.random() < 0.3:
                place, i, what, barriers = self.in_flight.pop(self.r.randrange(len(self.in_flight)))
                place[i] = what
                barriers[i].arrive()
                idle = 0
            warp = self.r.choice(warps)
            try:
                next(warp)
            except StopIteration:
                warps.remove(warp)
                idle = 0
            idle += 1
            need(idle < 20000, "nothing goes on")
        need(not self.in_flight, "copies in flight at the end")
        if not self.failed:
            need(len(self.put) == len(self.items) * self.RW, "results that were not put")


def breaks(shape, **kw):
    for seed in range(400):
        try:
            Cta(shape, seed, **kw).run()
        except Broken as e:
            return str(e)
    return None


@pytest.mark.parametrize("shape", shapes())
def test_every_shape(shape):
    warps, rw, feed, stages, slots = shape
    assert stages % (warps // rw) == 0 and stages % feed == 0 and stages > warps // rw
    for seed in range(25):
        Cta(shape, seed).run()


@pytest.mark.parametrize("shape", shapes())
@pytest.mark.parametrize("patience", [0.5, 0.02, 0.002])
def test_waits_that_run_out(shape, patience):
    """Nothing that is not there is read, and all copies have landed when the last warp ends."""
    failed = 0
    for seed in range(25):
        cta = Cta(shape, seed, patience=patience)
        cta.run()
        failed += cta.failed
    assert failed


def test_what_the_protocol_needs():
    """Without one of its parts the model breaks: the rings and turns are as they are for a reason."""
    assert breaks((8, 4, 2, 6, 2)) is None
    assert breaks((6, 2, 2, 8, 2)) is not None  # stages are no multiple of the key groups
    assert breaks((4, 1, 2, 9, 4)) is not None  # nor of the feeding warps
    assert breaks((4, 1, 2, 8, 4), without=("last join",)) is not None
    assert breaks((4, 1, 2, 8, 4), patience=0.05, without=("drain",)) == "copies in flight at the end"
