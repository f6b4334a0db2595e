"""A host model of the barriers of the 8-bit products' tensor-memory kernel (w8_linear_tc.cu), a CTA by itself and a pair,
explored over random interleavings, with waits that give up.

The model takes what the kernel does as atomic actions of a random scheduler, with its rings, counts of arrivals and orders:
  weights    copies weights of a step into a slot of its own ring, which the converters hand back
  tokens     copies tokens (a pair: of both CTAs, completing the first's barrier) into a step's slot, which the products
             hand back
  converters widen a step's weights into the step's slot and arrive (a pair: at the first CTA)
  products   waits for steps and drained accumulators, issues; what it issues is done later, in order, with its commits
  drains     take a finished accumulator and hand it back; a tile whose wait gave up is written as not a number
  copies     land at any time after they are issued, and within a wait's budget
A wait may give up, and then its CTA's other waits do; that CTA stays for the budget once all roles have ended.  Whatever
happens: every role ends, no barrier gets more arrivals than it counts, a tile is right or not a number, and nothing is on
its way to a CTA's shared memory when it ends, above all where none of its own waits gave up.
Without a wait that gives up every tile is right.  Mutants that the model must catch are at the end."""
import random

import pytest

SLOTS, RING, CHUNK, CONV, DRAINS = 4, 3, 3, 2, 2  # slots of steps and of weights, steps of an accumulator, warps


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = self.bytes = 0

    def arrive(self, n=1):
        assert 0 < n <= self.pending, "more arrivals than the barrier counts"
        self.pending -= n
        self._turn()

    def expect(self, n):
        self.bytes += n

    def complete(self, n):
        self.bytes -= n
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.pending = self.count
            self.phase += 1

    def done(self, parity):
        return (self.phase & 1) != parity


class Cta:
    def __init__(self, pair):
        n = 2 if pair else 1
        self.a8_full, self.a8_empty = [Barrier(1) for _ in range(RING)], [Barrier(CONV) for _ in range(RING)]
        self.full = [Barrier(CONV * n + 1) for _ in range(SLOTS)]
        self.empty = [Barrier(1) for _ in range(SLOTS)]
        self.acc_full, self.acc_empty = [Barrier(1) for _ in "ab"], [Barrier(DRAINS * n) for _ in "ab"]
        self.drain = Barrier(1)
        self.abort = self.ended = False
        self.weights, self.tokens = [None] * RING, [None] * SLOTS
        self.widened = [[None] * CONV for _ in range(SLOTS)]
        self.out = {}


class Kernel:
    OWN, OTHERS = 3, 5  # bytes of a step's tokens

    def __init__(self, pair, tiles, stages, rate, rng, mutant=None):
        self.pair, self.tiles, self.stages, self.rate, self.rng, self.mutant = pair, tiles, stages, rate, rng, mutant
        self.total = tiles * stages
        self.ctas = [Cta(pair) for _ in range(2 if pair else 1)]
        self.first = self.ctas[0]
        self.copies = []           # (cta, action at landing)
        self.queue = []            # of the tensor core
        self.acc = [[], []]        # steps that an accumulator has summed
        self.gave_up = self.force = False

    # ---- waits
    def wait(self, cta, bar, parity, last=False):
        """last: one that the abort flag does not cut short; only a copy or product that never ends would let it run out."""
        while not bar.done(parity):
            if not last and (cta.abort or self.force or self.rng.random() < self.rate):
                self.gave_up |= not cta.abort
                self.force = False
                cta.abort = True
                return False
            yield
        return True

    def copy(self, cta, owner, bar, size, action):
        """Into the CTA, completing a barrier of `owner`'s."""
        def land():
            assert not cta.ended and not owner.ended, "a copy lands in a CTA that has ended"
            action()
            bar.complete(size)
        self.copies.append(land)

    # ---- roles
    def weights(self, cta):
        s, ph, wrapped, ok = 0, 0, False, True
        for k in range(self.total):
            if wrapped and not (yield from self.wait(cta, cta.a8_empty[s], ph ^ 1)):
                break
            cta.a8_full[s].expect(4)
            cta.a8_full[s].arrive()
            self.copy(cta, cta, cta.a8_full[s], 4, lambda s=s, k=k: cta.weights.__setitem__(s, k))
            yield
            s += 1
            if s == RING:
                s, ph, wrapped = 0, ph ^ 1, True
        for i in range(RING):
            if i < s or wrapped:
                yield from self.wait(cta, cta.a8_full[i], ph if i < s else ph ^ 1, last=True)

    def tokens(self, cta):
        second = cta is not self.first
        s, ph, wrapped = 0, 0, False
        for k in range(self.total):
            if wrapped and not (yield from self.wait(cta, cta.empty[s], ph ^ 1)):
                break
            if not second:
                cta.full[s].expect(self.OWN + (self.OTHERS if self.pair else 0))
                cta.full[s].arrive()
                if self.rng.random() < 0.3:
                    yield
            self.copy(cta, self.first, self.first.full[s], self.OTHERS if second else self.OWN, lambda s=s, k=k: cta.tokens.__setitem__(s, k))
            yield
            s += 1
            if s == SLOTS:
                s, ph, wrapped = 0, ph ^ 1, True
        if self.mutant == "early" and cta.abort:
            self.budget()

    def budget(self):
        """Time in which everything that is on its way lands."""
        while self.copies:
            self.copies.pop(self.rng.randrange(len(self.copies)))()

    def convert(self, cta, w):
        s8, s, p8, ph, k, codes = 0, 0, 0, 0, 0, None

        def load():
            nonlocal s8, p8, codes
            if not (yield from self.wait(cta, cta.a8_full[s8], p8)):
                return False
            codes = cta.weights[s8]
            yield
            cta.a8_empty[s8].arrive()
            s8 += 1
            if s8 == RING:
                s8, p8 = 0, p8 ^ 1
            return True
        ok = self.total > 0 and (yield from load())
        while ok and k < self.total:
            if k >= SLOTS and not (yield from self.wait(cta, cta.empty[s], ph ^ 1)):
                break
            cta.widened[s][w] = codes
            yield
            if k + 1 < self.total:
                ok = yield from load()
            self.first.full[s].arrive()
            yield
            s += 1
            if s == SLOTS:
                s, ph = 0, ph ^ 1
            k += 1
    def issue(self, *what):
        self.queue.append(what)

    def products(self, cta):
        halves = 2 if self.pair else 1
        s, ph, chunk, ok, k = 0, 0, 0, True, 0
        for _ in range(self.tiles):
            kc, kb = 0, 0
            while ok and kb < self.stages:
                steps = 2 if halves == 2 and kc + 1 < CHUNK and kb + 1 < self.stages else 1
                last = kc + steps == CHUNK or kb + steps == self.stages
                for h in range(halves):
                    buf, used = (h, chunk) if halves == 2 else (chunk & 1, chunk >> 1)
                    if kc == 0 and used > 0:
                        ok = ok and (yield from self.wait(cta, cta.acc_empty[buf], (used - 1) & 1))
                    for i in range(steps):
                        at = (s + i) % SLOTS
                        if h == 0:
                            ok = ok and (yield from self.wait(cta, cta.full[at], ph if s + i < SLOTS else ph ^ 1))
                        if not ok:
                            break
                        self.issue("product", buf, at, k + i, kc + i == 0)
                        if h == halves - 1:
                            self.issue("commit", [c.empty[at] for c in self.ctas])
                        if last and i + 1 == steps:
                            self.issue("commit", [c.acc_full[buf] for c in self.ctas])
                        yield
                s += steps
                if s >= SLOTS:
                    s, ph = s - SLOTS, ph ^ 1
                kb += steps
                k += steps
                if last:
                    chunk, kc = chunk + 1, 0
                else:
                    kc += steps
            if not ok:
                break
        self.issue("commit", [c.drain for c in self.ctas])
        yield from self.wait(cta, cta.drain, 0, last=True)

    def products_of_second(self, cta):
        yield from self.wait(cta, cta.drain, 0, last=True)

    def tensor(self):
        """The next of what has been issued."""
        kind, *rest = self.queue.pop(0)
        if kind == "commit":
            for b in rest[0]:
                b.arrive()
            return
        buf, at, step, fresh = rest
        right = all(c.tokens[at] == step and c.widened[at] == [step] * CONV for c in self.ctas)
        self.acc[buf] = ([] if fresh else self.acc[buf]) + [step if right else None]

    def drains(self, cta, w):
        halves = 2 if self.pair else 1
        chunk, ok = 0, True
        for tile in range(self.tiles):
            sums = [[] for _ in range(halves)]
            for kb in range(0, self.stages, CHUNK):
                if not ok:
                    break
                for h in range(halves):
                    buf, used = (h, chunk) if halves == 2 else (chunk & 1, chunk >> 1)
                    ok = ok and (yield from self.wait(cta, cta.acc_full[buf], used & 1))
                    if not ok:
                        break
                    sums[h] += self.acc[buf]
                    yield
                    self.first.acc_empty[buf].arrive()
                    yield
                chunk += 1
            cta.out[tile, w] = sums if ok or self.mutant == "sums" else None

    def run(self):
        actors = []
        for c in self.ctas:
            actors += [self.weights(c), self.tokens(c), (self.products if c is self.first else self.products_of_second)(c)]
            actors += [self.convert(c, w) for w in range(CONV)] + [self.drains(c, w) for w in range(DRAINS)]
        self._finish(actors)
        for c in self.ctas:  # those that do not wait end at once
            c.ended = not c.abort or self.mutant in ("leave", "early")
        self.budget()

    def _finish(self, actors):
        idle = 0
        while actors:
            i = self.rng.randrange(len(actors) + 2)
            if i >= len(actors):
                if i == len(actors) and self.copies and self.rng.random() < 0.5:
                    self.copies.pop(self.rng.randrange(len(self.copies)))()
                    idle = 0
                elif self.queue and self.rng.random() < 0.5:
                    self.tensor()
                    idle = 0
                continue
            before = self.state()
            try:
                next(actors[i])
            except StopIteration:
                del actors[i]
            idle = 0 if self.state() != before else idle + 1
            if idle > 400 and not self.copies and not self.queue:
                assert idle < 2000, "a role that does not end"
                if self.gave_up:  # the other CTA of one that gave up: its waits run out
                    self.force = True

    def state(self):
        return (len(self.copies), len(self.queue), [[(b.phase, b.pending, b.bytes) for b in c.a8_empty + c.a8_full + c.full + c.acc_empty]
                                                    for c in self.ctas], [c.abort for c in self.ctas])

    def check(self):
        nans = 0
        for c in self.ctas:
            for tile in range(self.tiles):
                want = list(range(tile * self.stages, (tile + 1) * self.stages))
                for w in range(DRAINS):
                    got = c.out[tile, w]
                    nans += got is None
                    assert got is None or got == [want] * len(got), "a wrong sum that is not marked"
        assert not nans or self.gave_up
        return nans


def explore(pair, rate, seeds, mutant=None):
    nans = left = 0
    for seed in range(seeds):
        rng = random.Random(seed * 7 + pair)
        k = Kernel(pair, rng.randint(1, 3), rng.randint(1, 8), rng.choice(rate), rng, mutant)
        k.run()
        nans += k.check()
        left += any(c.abort for c in k.ctas)
    return nans, left


@pytest.mark.parametrize("pair", [False, True])
def test_every_tile_is_right_without_a_wait_that_gives_up(pair):
    assert explore(pair, [0.0], 120) == (0, 0)


@pytest.mark.parametrize("pair", [False, True])
def test_waits_that_give_up(pair):
    nans, left = explore(pair, [0.0003, 0.003, 0.03], 500)
    assert nans > 100 and left > 100  # both are met


@pytest.mark.parametrize("mutant, pair, says", [
    ("leave", False, "has ended"), ("leave", True, "has ended"),  # a CTA ends without waiting for its copies
    ("early", True, "has ended"),                                 # it waits when the copying role ends, not the others
    ("sums", False, "not marked"), ("sums", True, "not marked")])  # a tile whose wait gave up is written all the same
def test_mutants_are_caught(mutant, pair, says):
    with pytest.raises(AssertionError, match=says):
        explore(pair, [0.0003, 0.003, 0.03], 500, mutant)


def test_the_kernel_waits_for_copies_after_its_roles():
    """What the model takes from the source: past the last barrier of all roles, by the abort flag alone."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"//[^\n]*", "", open(os.path.join(root, "moe_expert_ffn_dispatch_gb300", "csrc", "w8_linear_tc.cu")).read())
    call = re.search(r"if \(FORM != kFew && warp == 2 && \*abort\) wait_out_budget\(\);", src)
    assert call and src.rindex("wait(&bar") < src.rindex("if constexpr (FORM == kTwo) cluster_sync();", 0, call.start())
    assert src.count("wait_out_budget()") == 2  # the function and its call
