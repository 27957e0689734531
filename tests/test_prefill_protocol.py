"""Model of the barrier protocol of the prefill kernel
(csrc/pa_prefill_umma.cuh), run under random schedules on the CPU.

Roles of a CTA: copiers (one per unit of a tile for quantised D = 256, else
one) fill units of a ring in the order K, V interleaved; MMA warps (one per
row tile at D = 128, one at D = 256) issue S = Q K and O += P V, which an
engine per warp retires in order, commits included; two softmax groups per
row tile read their half of S, agree on a new maximum (named barrier), may
rescale O, and write P over S.  Three forms: D = 128 ("d128"), D = 128 with
the halves of S taking turns ("turns": no maximum, no agreement) and D = 256
("d256", two S buffers).

The asserts check the data flow: no unit refilled before its readers are
complete, no S written over weights still to be read, no O rescaled while a
product is in flight, nothing read before it is written.  With an expired
wait the data are void, and the model checks that every role still ends with
every barrier between warps met and nothing in flight."""
import random

import pytest

from tests.test_verify_protocol import Bar

FORMS = ["d128", "turns", "d256"]


class Prefill:
    def __init__(self, form, tiles, quant, row_tiles=2, rescale=0.3):
        self.form, self.n, self.d256 = form, tiles, form == "d256"
        self.H = 2 if self.d256 else 1
        self.RT = 1 if self.d256 else row_tiles
        self.NU = 4 if quant else 5
        self.copiers = self.H if quant else 1
        self.rescale = rescale
        self.full = [Bar(1) for _ in range(self.NU)]
        self.empty = [Bar(self.RT) for _ in range(self.NU)]
        turns = form == "turns"
        self.sfull = [Bar(1) for _ in range(4)]
        self.pready = [Bar(1 if turns else 2) for _ in range(4)]
        self.odone = [Bar(1) for _ in range(2)]
        self.done = Bar(self.RT)
        self.unit = [None] * self.NU
        self.readers = [0] * self.NU
        self.s = {}            # (row tile, buffer, half) -> ("S" | "P", tile) or None
        self.issued = {}       # row tile -> products of PV issued, retired
        self.queue = [[] for _ in range(self.RT)]
        self.votes, self.abort, self.expire = {}, False, None

    # ---- waits
    def wait(self, bar, parity):
        if self.expire is not None and not bar.ready(parity):
            self.expire -= 1
            if self.expire < 0:
                self.expire, self.abort = None, True
        while not bar.ready(parity) and not self.abort:
            yield lambda: bar.ready(parity) or self.abort

    def meet(self, key):   # named barrier of a pair: no abort ends it
        self.votes[key] = self.votes.get(key, 0) + 1
        while self.votes[key] < 2:
            yield lambda: self.votes[key] >= 2

    def check(self, ok, what):
        assert ok or self.abort, what

    # ---- roles
    def order(self):
        """(is_v, tile): K runs one tile (D = 128) or two (D = 256) ahead of V."""
        for q in range(2 * self.n + 1):
            if self.d256:
                v = q > 0 and q % 2 == 0
                j = q // 2 - 1 if v else (q + 1) // 2
            else:
                v, j = q % 2 == 1, q // 2
            if j < self.n:
                yield v, j

    def copier(self, c):
        u = c
        for v, j in self.order():
            for h in range(self.H) if self.copiers == 1 else [c]:
                st = u % self.NU
                if u >= self.NU:
                    yield from self.wait(self.empty[st], (u // self.NU - 1) & 1)
                self.check(self.readers[st] == 0, "unit refilled while it is read")
                self.unit[st], self.readers[st] = (v, j, h), self.RT
                self.full[st].arrive()
                u += 1 if self.copiers == 1 else self.H
                yield None

    def qk(self, t, u, j, h, buf, halves):
        def retire():
            st = u % self.NU
            self.check(self.unit[st] == (False, j, h), "Q K of another unit")
            for x in halves:
                self.check(h > 0 or self.s.get((t, buf, x)) is None, "S over unread weights")
                self.s[t, buf, x] = ("S", j)
        self.queue[t].append(retire)

    def pv(self, t, u, j, h, buf, halves, last):
        self.issued.setdefault(t, [0, 0])[0] += 1

        def retire():
            st = u % self.NU
            self.check(self.unit[st] == (True, j, h), "P V of another unit")
            for x in halves:
                self.check(self.s.get((t, buf, x)) == ("P", j), "P V before its weights")
                if last:
                    self.s[t, buf, x] = None
            self.issued[t][1] += 1
        self.queue[t].append(retire)

    def commit(self, t, bar, frees=None):
        def retire():
            if frees is not None:
                self.readers[frees] -= 1
            bar.arrive()
        self.queue[t].append(retire)

    def free(self, t, u):
        self.commit(t, self.empty[u % self.NU], u % self.NU)

    def fbar(self, u):
        return self.full[u % self.NU], (u // self.NU) & 1

    def mma(self, t):
        n = self.n
        if self.d256:
            u = 0

            def tile(j):
                nonlocal u
                for h in range(2):
                    yield from self.wait(*self.fbar(u))
                    self.qk(t, u, j, h, j & 1, (0, 1))
                    self.free(t, u)
                    u += 1
                self.commit(t, self.sfull[j & 1])
            for j in range(min(2, n)):
                yield from tile(j)
            for j in range(n):
                yield from self.wait(*self.fbar(u))
                yield from self.wait(self.pready[j & 1], (j >> 1) & 1)
                for h in range(2):
                    if h:
                        yield from self.wait(*self.fbar(u))
                    self.pv(t, u, j, h, j & 1, (0, 1), h == 1)
                    self.free(t, u)
                    u += 1
                self.commit(t, self.odone[j & 1])
                if j + 2 < n:
                    yield from tile(j + 2)
        elif self.form == "turns":
            def half(u, j, x):
                self.qk(t, u, j, 0, 0, (x,))
                self.commit(t, self.sfull[2 * t + x])
            if n:
                yield from self.wait(*self.fbar(0))
                half(0, 0, 0)
                half(0, 0, 1)
                self.free(t, 0)
            for j in range(n):
                uv, uk = 2 * j + 1, 2 * j + 2
                yield from self.wait(*self.fbar(uv))
                for x in range(2):
                    yield from self.wait(self.pready[2 * t + x], j & 1)
                    self.pv(t, uv, j, 0, 0, (x,), True)
                    if x:
                        self.free(t, uv)
                    if j + 1 < n:
                        if not x:
                            yield from self.wait(*self.fbar(uk))
                        half(uk, j + 1, x)
                        if x:
                            self.free(t, uk)
            if n:
                self.commit(t, self.odone[t])
        else:
            if n:
                yield from self.wait(*self.fbar(0))
                self.qk(t, 0, 0, 0, 0, (0, 1))
                self.commit(t, self.sfull[t])
                self.free(t, 0)
            for j in range(n):
                uv, uk = 2 * j + 1, 2 * j + 2
                yield from self.wait(*self.fbar(uv))
                yield from self.wait(self.pready[t], j & 1)
                self.pv(t, uv, j, 0, 0, (0, 1), True)
                self.free(t, uv)
                if j + 1 == n:
                    break
                yield from self.wait(*self.fbar(uk))
                self.qk(t, uk, j + 1, 0, 0, (0, 1))
                self.commit(t, self.sfull[t])
                self.free(t, uk)
            if n:
                self.commit(t, self.odone[t])
        self.commit(t, self.done)
        while not self.done.ready(0):      # (drained whatever happened)
            yield lambda: self.done.ready(0)

    def softmax(self, t, x, rng):
        n = self.n
        for j in range(n):
            buf = j & 1 if self.d256 else 0
            turn = 2 * t + x if self.form == "turns" else (buf if self.d256 else t)
            yield from self.wait(self.sfull[turn], ((j >> 1) if self.d256 else j) & 1)
            self.check(self.s.get((t, buf, x)) == ("S", j), "S read before it is there")
            yield None
            if self.form != "turns":
                yield from self.meet((t, j, "vote"))
                if random.Random(self.seed * 1000 + t * 100 + j).random() < self.rescale:
                    yield from self.meet((t, j, "a"))
                    yield from self.meet((t, j, "b"))
                    if j:
                        if self.d256:
                            yield from self.wait(self.odone[(j - 1) & 1], ((j - 1) >> 1) & 1)
                        a, b = self.issued.get(t, (0, 0))
                        self.check(a == b == j * self.H, "O rescaled under a product")
            self.s[t, buf, x] = ("P", j)
            self.pready[turn].arrive()
        for k in "abc":
            yield from self.meet((t, "end", k))
        if n:
            last = (n - 1) & 1 if self.d256 else t
            yield from self.wait(self.odone[last], ((n - 1) >> 1) & 1 if self.d256 else 0)
            per = 2 if self.d256 or self.form == "turns" else 1
            self.check(self.issued[t][1] == n * per, "output before the last product")
            if not self.d256 and self.RT == 2:   # fp32 rows take the other row tile's queries' place
                yield from self.wait(self.odone[t ^ 1], 0)
                self.check(self.issued[t ^ 1][1] == n * per, "queries overwritten under their products")

    def run(self, seed, expire=None):
        self.seed, self.expire = seed, expire
        rng = random.Random(seed)
        roles = [self.copier(c) for c in range(self.copiers)] + [self.mma(t) for t in range(self.RT)]
        roles += [self.softmax(t, x, rng) for t in range(self.RT) for x in range(2)]
        blocked = [None] * len(roles)
        alive = set(range(len(roles)))
        idle = 0
        while alive:
            progress = False
            for a in rng.sample(sorted(alive), rng.randint(1, len(alive))):
                if blocked[a] is not None and not blocked[a]():
                    continue
                try:
                    blocked[a] = next(roles[a])
                except StopIteration:
                    alive.discard(a)
                progress = True
            for q in self.queue:
                if q and rng.random() < 0.5:
                    q.pop(0)()
                    progress = True
            idle = 0 if progress or any(self.queue) else idle + 1
            assert idle < 50, f"deadlock: {sorted(alive)}"
        assert not any(self.queue), "products in flight at the end"
        assert all(v == 2 for v in self.votes.values())


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n", [0, 1, 2, 3, 4, 7, 12])
def test_random_schedules(form, n, quant):
    for seed in range(25):
        for rt in (1, 2):
            Prefill(form, n, quant, rt).run(seed)


@pytest.mark.parametrize("form", FORMS)
def test_an_expired_wait_ends_every_role(form):
    for seed in range(60):
        for quant in (False, True):
            Prefill(form, 6, quant).run(seed, expire=seed % 30)


@pytest.mark.parametrize("form,method", [("d128", "empty"), ("d256", "odone"), ("turns", "pready"), ("turns", "odone")])
def test_the_model_catches_a_missing_wait(form, method):
    class Broken(Prefill):
        def wait(self, bar, parity):
            if bar not in getattr(self, method):
                yield from super().wait(bar, parity)

    with pytest.raises(AssertionError):
        for seed in range(80):
            Broken(form, 8, False, rescale=0.8).run(seed)
