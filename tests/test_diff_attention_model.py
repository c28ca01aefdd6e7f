"""The differential attention kernel's work list and synchronisation, restated and checked on the CPU.

Work items: item w is head w % heads of query tile w // heads, and row r's tiles start at number
cu[r] // 128 + r; no table is built.  Every tile of every row must be found exactly once, whatever the
lengths, by the 32-probe search that the kernel runs.

Synchronisation: the roles of `k_diff_attention` (csrc/diff_attention.cu) - the TMA producer, the warp that
finishes an item's last V tile, one MMA thread a map, a softmax group a map, and the read-out - meet only on
mbarriers.  The model below states each role's waits and arrivals in the kernel's
order; mbarrier waits go by phase parity, exactly as on the device, so that a wait which could take one phase
for another shows up.  Random interleavings must finish, no wait may pass on a phase that is not the one it
means, and no buffer may be refilled before its readers are done.  Planted errors in the model must be caught.
"""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "encoder_decision_model_b200", "csrc", "diff_attention.cu")


def find_row(starts, b):
    """The kernel's search: the last r with starts[r] <= b, 32 probes at a time; None if there is none."""
    lo, n = 0, len(starts)
    while n > 1:
        step = (n + 31) >> 5
        below = [i for i in range(32) if i * step < n and starts[lo + i * step] <= b]
        if 0 not in below:
            return None
        k = max(below)
        lo += k * step
        n = min(step, n - k * step)
    return lo


@pytest.mark.parametrize("tile", [128, 64, 32])
def test_every_query_tile_is_found_once(tile):
    rng = random.Random(1)
    for case in range(300):
        n = rng.choice([1, 2, 5, 31, 32, 33, 200, 1100])
        top = rng.choice([1, 3, tile, 3 * tile, 700])
        lens = [rng.choice([0, rng.randint(0, top), tile, tile + 1, tile - 1]) for _ in range(n)]
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        T = cu[-1] + rng.choice([0, 7, 300])  # tokens behind the last row
        starts = [cu[r] // tile + r for r in range(n)]
        found = []
        for b in range(T // tile + n):
            r = find_row(starts, b)
            if r is None:
                continue
            q0 = cu[r] + (b - starts[r]) * tile
            if cu[r] <= q0 < cu[r + 1]:
                found.append(q0)
        want = [a + i for a, x in zip(cu, lens) for i in range(0, x, tile)]
        assert found == want, (lens, found, want)


# ------------------------------------------------------------------ synchronisation


class Bar:
    """mbarrier: `count` arrivals complete a phase.  `expect` counts TMA bytes as one more pending arrival."""

    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        assert self.pending > 0
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passes(self, parity):
        return (self.phase - 1) & 1 == parity and self.phase > 0 or (self.phase == 0 and parity == 1)


class Model:
    def __init__(self, items, seed, plant=None, NK=8, NV=4):
        self.items, self.plant, self.NK, self.NV = items, plant, NK, NV
        self.rng = random.Random(seed)
        B = Bar
        self.qfull, self.qfree = [B(1), B(1)], [B(2), B(2)]
        self.kfull, self.kfree = [B(1) for _ in range(NK)], [B(1) for _ in range(NK)]
        self.vfull, self.vfree = [B(1) for _ in range(NV)], [B(2) for _ in range(NV)]
        self.vtail = [B(1) for _ in range(NV)]
        self.sfull, self.pready, self.pvdone = ([B(1) for _ in range(4)] for _ in range(3))
        # (one arrival on pready or summed stands for a group's four warps, one on ofree for the read-out's)
        self.odone, self.summed, self.ofree = [B(1), B(1)], [B(2), B(2)], B(1)
        self.sums = [[None, None], [None, None]]
        self.k, self.v, self.q, self.s = {}, {}, {}, {}  # what each buffer holds: a tag
        self.async_ops = []  # TMA loads and MMA completions, finishing in any order that the hardware allows
        self.o_owner = [None, None]

    def wait(self, bar, parity, meant):
        """Blocks until the parity test passes; then the phase must be the one meant."""
        while not bar.passes(parity):
            yield
        assert bar.phase >= meant + 1, "a wait passed on another phase"
        assert bar.phase <= meant + 2 and (bar.phase == meant + 1 or not self.strict(bar)), "a phase was missed"

    def strict(self, bar):
        return True

    # -- roles
    def producer(self):
        c = 0
        for it, nt_tail in enumerate(self.items):
            nt, tail = nt_tail
            buf = it & 1
            if it >= 2:
                yield from self.wait(self.qfree[buf], ((it - 2) >> 1) & 1, (it - 2) >> 1)
            self.load(self.q, buf, ("q", it), self.qfull[buf])
            for j in range(nt):
                for x in (0, 1):
                    u = 2 * c + x
                    s = u % self.NK
                    if u >= self.NK:
                        yield from self.wait(self.kfree[s], ((u - self.NK) // self.NK) & 1, (u - self.NK) // self.NK)
                    self.load(self.k, s, ("k", c, x), self.kfull[s])
                    yield
                s = c % self.NV
                if c >= self.NV:
                    yield from self.wait(self.vfree[s], ((c - self.NV) // self.NV) & 1, (c - self.NV) // self.NV)
                last = j == nt - 1 and tail
                self.load(self.v, s, ("raw" if last else "v", c), self.vtail[s] if last else self.vfull[s])
                yield
                c += 1

    def load(self, where, slot, tag, bar):
        def done():
            where[slot] = tag
            bar.arrive()
        self.async_ops.append(done)

    def fixer(self):
        c, tails = 0, [0] * self.NV
        for nt, tail in self.items:
            c += nt
            if not tail:
                continue
            s = (c - 1) % self.NV
            if self.plant == "tail":  # waits for the stage's phase instead of its own barrier
                yield from self.wait(self.vfull[s], ((c - 1) // self.NV) & 1, (c - 1) // self.NV)
            else:
                yield from self.wait(self.vtail[s], tails[s] & 1, tails[s])
            tails[s] += 1
            assert self.v[s] == ("raw", c - 1)
            self.v[s] = ("v", c - 1)
            self.vfull[s].arrive()
            yield

    def mma(self, x):
        s_queue, pv_queue = self.mma_queue[2 * x], self.mma_queue[2 * x + 1]  # no order between the two is relied on
        sc = c = 0
        ahead = 0
        n = len(self.items)

        def issue_s(it, j, last):
            nonlocal sc
            b, u = 2 * x + (sc & 1), 2 * sc + x
            s = u % self.NK
            yield from self.wait(self.kfull[s], (u // self.NK) & 1, u // self.NK)
            if sc >= 2 and self.plant != "overlay":
                yield from self.wait(self.pvdone[b], ((sc - 2) >> 1) & 1, (sc - 2) >> 1)
            t, buf = sc, it & 1

            def run():
                assert self.q[buf] == ("q", it) and self.k[s] == ("k", t, x)
                assert self.s.get(b) in (None, ("used", t - 2)), "S written over P that is still needed"
                self.s[b] = ("s", t)
                self.sfull[b].arrive()
                self.kfree[s].arrive()
                if last:
                    self.qfree[buf].arrive()
            s_queue.append(run)
            sc += 1

        for it, (nt, _) in enumerate(self.items):
            if ahead == 0:
                yield from self.wait(self.qfull[it & 1], (it >> 1) & 1, it >> 1)
            while ahead < min(2, nt):
                ahead += 1
                yield from issue_s(it, ahead - 1, ahead == nt)
            nahead = 0
            for j in range(nt):
                b, s = 2 * x + (c & 1), c % self.NV
                yield from self.wait(self.vfull[s], (c // self.NV) & 1, c // self.NV)
                yield from self.wait(self.pready[b], (c >> 1) & 1, c >> 1)
                if j == 0 and it > 0 and self.plant != "ofree":
                    yield from self.wait(self.ofree, (it - 1) & 1, it - 1)
                t, first, last = c, j == 0, j == nt - 1

                def run(b=b, s=s, t=t, first=first, last=last, it=it):
                    assert self.v[s] == ("v", t) and self.s[b] == ("p", t)
                    if first:
                        assert self.o_owner[x] in (None, ("read", it - 1)), "O overwritten before it was read"
                        self.o_owner[x] = ("acc", it)
                    assert self.o_owner[x] == ("acc", it)
                    self.s[b] = ("used", t)
                    self.pvdone[b].arrive()
                    self.vfree[s].arrive()
                    if last:
                        self.odone[x].arrive()
                pv_queue.append(run)
                c += 1
                if ahead < nt:
                    ahead += 1
                    yield from issue_s(it, ahead - 1, ahead == nt)
                elif it + 1 < n and nahead < min(2, self.items[it + 1][0]):
                    if nahead == 0:
                        yield from self.wait(self.qfull[(it + 1) & 1], ((it + 1) >> 1) & 1, (it + 1) >> 1)
                    nahead += 1
                    yield from issue_s(it + 1, nahead - 1, nahead == self.items[it + 1][0])
                yield
            ahead = nahead

    def softmax(self, x):
        c = 0
        for it, (nt, _) in enumerate(self.items):
            for j in range(nt):
                b = 2 * x + (c & 1)
                yield from self.wait(self.sfull[b], (c >> 1) & 1, c >> 1)
                assert self.s[b] == ("s", c)
                yield
                if j and self.rng.random() < 0.3:  # a running maximum moves: O has to be at rest
                    o = 2 * x + ((c - 1) & 1)
                    yield from self.wait(self.pvdone[o], ((c - 1) >> 1) & 1, (c - 1) >> 1)
                self.s[b] = ("p", c)
                self.pready[b].arrive()
                c += 1
                yield
            self.sums[it % self.kept][x] = it
            self.summed[it & 1].arrive()
            yield

    def readout(self):
        for it in range(len(self.items)):
            yield from self.wait(self.summed[it & 1], (it >> 1) & 1, it >> 1)
            for m in (0, 1):
                yield from self.wait(self.odone[m], it & 1, it)
            yield
            assert self.sums[it % self.kept] == [it, it], "the sums of another item"
            assert self.o_owner == [("acc", it)] * 2
            self.o_owner = [("read", it)] * 2
            self.ofree.arrive()
            yield

    def run(self):
        self.mma_queue = [[] for _ in range(4)]
        self.kept = 1 if self.plant == "sums" else 2  # items whose sums are kept
        roles = [self.producer(), self.fixer(), self.mma(0), self.mma(1), self.softmax(0), self.softmax(1), self.readout()]
        speed = [self.rng.choice([1, 4, 60]) for _ in roles]  # some roles far slower than others
        idle = 0
        while roles:
            k = self.rng.choices(range(len(roles) + 2), speed + [8, 8])[0]
            before = len(roles)
            if k < len(roles):
                try:
                    next(roles[k])
                except StopIteration:
                    roles.pop(k)
                    speed.pop(k)
            elif k == len(roles) and self.async_ops:  # loads land in any order
                self.async_ops.pop(self.rng.randrange(len(self.async_ops)))()
                idle = 0
            else:  # a map's S products run in order, and its PV products
                for q in self.rng.sample(self.mma_queue, 4):
                    if q:
                        q.pop(0)()
                        idle = 0
                        break
            idle += 1
            assert idle < 20000, "no role can go on"
            if before != len(roles):
                idle = 0


def _items(rng):
    return [(rng.choice([1, 1, 2, 3, 4, 9]), rng.random() < 0.6) for _ in range(rng.randint(1, 12))]


def test_random_interleavings_finish_in_order():
    for seed in range(150):
        rng = random.Random(seed)
        Model(_items(rng), seed).run()


@pytest.mark.parametrize("plant", ["tail", "overlay", "ofree", "sums"])
def test_planted_errors_are_caught(plant):
    caught = 0
    for seed in range(150):
        rng = random.Random(1000 + seed)
        items = [(rng.choice([1, 1, 1, 2, 5, 6, 9]), True) for _ in range(10)]
        try:
            Model(items, seed, plant).run()
        except AssertionError:
            caught += 1
    assert caught > 0


def test_model_matches_the_source():
    src = open(SRC).read()
    assert re.search(r"NK = (\d+), NV = (\d+);", src).groups() == ("8", "4")
    for name, count in (("vfree", 2), ("qfree", 2), ("vtail", 1), ("odone", 1), ("pready", 4), ("pvdone", 1), ("sfull", 1), ("summed", 8)):
        assert f"mbar_init(&{name}[i], {count});" in src, name
    assert "mbar_init(ofree, 4);" in src and "sums + 256 * (it & 1)" in src
    assert "j == t.nt - 1 && (t.in_last() & 15) ? &vtail[s] : &vfull[s]" in src
    assert "mbar_wait(&vtail[s], tails[s]++ & 1, status);" in src
    assert "if (sc >= 2) wait(b_pvdone + 8 * b, ((sc - 2) >> 1) & 1, status);" in src
