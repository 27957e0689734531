"""Models of the barrier protocols of the latent-attention kernels, run under
random schedules on the CPU.

Rows (csrc/pa_latent_rows.cu): a worker's run of pieces, each a number of key
tiles, each piece twice in the run that looks for maxima first.  Roles: one
copier (bf16) or two that take turns at the tiles (FP8), the queries' copier,
a warp for S = Q K and one for O += P V, each with an engine that retires its
products and commits in order, two softmax warps (of the four).

Prefill (csrc/pa_latent_prefill.cu): a stream of items of two row tiles that
share eight units of K (three a tile) and V (two), S of the two taking turns, the
second one seeing more tiles than the first; the output takes the queries' place.

The asserts check the data flow (nothing refilled, overwritten or read before
its time); with an expired wait the data are void, and the model checks that
every role ends with every barrier between warps met and nothing in flight."""
import random

import pytest

from tests.test_verify_protocol import Bar


class Model:
    def start(self, seed, expire):
        self.abort, self.expire, self.votes = False, expire, {}
        self.rng = random.Random(seed)

    def wait(self, bar, phase):
        """The wait for a barrier's phase-th completion, by its parity alone."""
        parity = phase & 1
        if self.expire is not None and not bar.ready(parity):
            self.expire -= 1
            if self.expire < 0:
                self.expire, self.abort = None, True
        while not bar.ready(parity) and not self.abort:
            yield lambda: bar.ready(parity) or self.abort

    def meet(self, key, n):   # named barrier: no abort ends it
        self.votes[key] = self.votes.get(key, 0) + 1
        while self.votes[key] < n:
            yield lambda: self.votes[key] >= n

    def drain(self, bar):
        while not bar.ready(0):
            yield lambda: bar.ready(0)

    def check(self, ok, what):
        assert ok or self.abort, what

    def play(self, roles):
        rng, blocked, alive, idle = self.rng, [None] * len(roles), set(range(len(roles))), 0
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


class Rows(Model):
    WARPS = 2

    def __init__(self, pieces, fp8=False, safe=False, stages=4, early_q=True):
        self.pieces, self.fp8, self.safe, self.NS, self.early_q = pieces, fp8, safe, stages, early_q
        self.full = [Bar(1) for _ in range(stages)]
        self.empty = [Bar(1) for _ in range(stages)]
        w = self.WARPS
        self.sfull, self.odone = [Bar(1) for _ in range(2)], [Bar(1) for _ in range(2)]
        self.sread, self.pready = [Bar(w) for _ in range(2)], [Bar(w) for _ in range(2)]
        self.qfull, self.qready, self.qfree, self.done = Bar(1), Bar(w), Bar(w), Bar(2)
        self.stage, self.readers = [None] * stages, [0] * stages
        self.s, self.p, self.o = [None, None], [None, None], None
        self.qsmem, self.qtmem = None, [None] * w
        self.pv_issued = self.pv_done = 0
        self.queue = [[], []]

    def tiles(self):
        """(piece, k, number): k < 0 the tiles of the run for the maximum."""
        g = 0
        for i, n in enumerate(self.pieces):
            for k in range(-n if self.safe else 0, n):
                yield i, k, g
                g += 1

    def copier(self, which, of):
        for i, k, g in self.tiles():
            if g % of != which:
                continue
            st = g % self.NS
            if g >= self.NS:
                yield from self.wait(self.empty[st], g // self.NS - 1)
            if self.abort and not self.fp8:
                return
            self.check(self.readers[st] == 0, "stage refilled while it is read")
            self.stage[st], self.readers[st] = g, 2
            self.full[st].arrive()
            yield None

    def query(self):
        for i in range(len(self.pieces)):
            if i:
                yield from self.wait(self.qfree, i - 1)
                if self.abort:
                    return
            self.qsmem = i
            self.qfull.arrive()
            yield None

    def scores(self):
        last = None
        for i, k, g in self.tiles():
            if i != last:
                yield from self.wait(self.qready, i)
                last = i
            if g >= 2:
                yield from self.wait(self.sread[g & 1], g // 2 - 1)
            yield from self.wait(self.full[g % self.NS], g // self.NS)

            def retire(i=i, g=g):
                self.check(self.stage[g % self.NS] == g, "S of another tile")
                self.check(all(q == i for q in self.qtmem), "S of other queries")
                self.check(self.early_q or self.qsmem == i, "S of other queries in shared memory")
                self.check(self.s[g & 1] in (None, ("read", g - 2)), "S over unread scores")
                self.s[g & 1] = ["there", g, 0]
                self.readers[g % self.NS] -= 1
                self.sfull[g & 1].arrive()
            self.queue[0].append(retire)
            yield None
        self.queue[0].append(self.done.arrive)
        yield from self.drain(self.done)

    def output(self):
        for i, k, g in self.tiles():
            yield from self.wait(self.full[g % self.NS], g // self.NS)
            yield from self.wait(self.pready[g & 1], g // 2)
            self.pv_issued += 1

            def retire(i=i, k=k, g=g):
                self.check(self.stage[g % self.NS] == g, "O of another tile")
                if k >= 0:
                    self.check(self.p[g & 1] == [g] * self.WARPS, "O before its weights")
                    self.check((self.o is None) if k == 0 else self.o == (i, k - 1), "O of another piece")
                    self.o = (i, k)
                self.readers[g % self.NS] -= 1
                self.pv_done += 1
                self.empty[g % self.NS].arrive()
                self.odone[g & 1].arrive()
            self.queue[1].append(retire)
            yield None
        self.queue[1].append(self.done.arrive)
        yield from self.drain(self.done)

    def softmax(self, w):
        last, count = None, 0
        order = list(self.tiles())
        for x, (i, k, g) in enumerate(order):
            if i != last:
                yield from self.wait(self.qfull, i)
                self.check(self.qsmem == i, "other queries")
                self.qtmem[w] = i
                self.qready.arrive()
                if self.early_q:
                    self.qfree.arrive()
                last = i
            yield from self.wait(self.sfull[g & 1], g // 2)
            yield from self.wait(self.full[g % self.NS], g // self.NS)
            s = self.s[g & 1]
            self.check(isinstance(s, list) and s[1] == g, "scores read before they are there")
            if isinstance(s, list):
                s[2] += 1
                if s[2] == self.WARPS:
                    self.s[g & 1] = ("read", g)
            self.sread[g & 1].arrive()
            yield None
            if g >= 2:
                yield from self.wait(self.odone[g & 1], g // 2 - 1)
            if k >= 0:
                if self.p[g & 1] is None or self.p[g & 1][w] != g:
                    self.p[g & 1] = list(self.p[g & 1] or [None] * self.WARPS)
                    self.p[g & 1][w] = g
            self.check(self.pv_done >= g - 1, "weights over those of an open product")
            self.pready[g & 1].arrive()
            yield None
            if x + 1 == len(order) or order[x + 1][0] != i:   # the end of a piece
                if not self.early_q:
                    self.qfree.arrive()
                yield from self.wait(self.odone[g & 1], g // 2)
                yield from self.meet((i, "sums"), self.WARPS)
                self.check(self.o == (i, k), "output before the last product")
                yield from self.meet((i, "written"), self.WARPS)
                self.o = None

    def run(self, seed, expire=None):
        self.start(seed, expire)
        of = 2 if self.fp8 else 1
        self.play([self.copier(c, of) for c in range(of)] + [self.query(), self.scores(), self.output()]
                  + [self.softmax(w) for w in range(self.WARPS)])


PIECES = [[1], [2], [5], [1, 1, 1], [3, 1, 7], [2, 6], []]


@pytest.mark.parametrize("pieces", PIECES)
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_random_schedules(pieces, fp8):
    for seed in range(40):
        for safe in (False, True):
            Rows(pieces, fp8, safe, stages=4 + seed % 2, early_q=seed % 3 > 0).run(seed)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_an_expired_wait_ends_every_role(fp8):
    for seed in range(80):
        Rows([3, 1, 6], fp8, seed % 2 == 0).run(seed, expire=seed % 25)


@pytest.mark.parametrize("method", ["empty", "sread", "odone", "pready", "qready"])
def test_rows_the_model_catches_a_missing_wait(method):
    class Broken(Rows):
        def wait(self, bar, phase):
            b = getattr(self, method)
            if bar not in (b if isinstance(b, list) else [b]):
                yield from super().wait(bar, phase)

    with pytest.raises(AssertionError):
        for seed in range(120):
            Broken([4, 3], early_q=True).run(seed)


class Prefill(Model):
    """A stream of items (key tiles of row tile 0, of row tile 1 or None, wide output)."""
    NU, PER, SLOTS = 8, 5, 4

    def __init__(self, items):
        self.items = items
        self.all = [max(n0, n1 or 0) for n0, n1, _ in items]
        self.full = [Bar(1) for _ in range(self.NU)]
        self.empty = [Bar(2) for _ in range(self.NU)]
        self.qfull, self.qfree, self.sfull, self.pready, self.odone = ([Bar(c) for _ in range(2)] for c in (1, 2, 1, 2, 1))
        self.ifull, self.iempty = ([Bar(c) for _ in range(self.SLOTS)] for c in (1, 6))
        self.done = Bar(2)
        self.unit, self.readers = [None] * self.NU, [0] * self.NU
        self.item = [None] * self.SLOTS
        self.q = [None, None]                       # item whose queries (or "out": output) are there
        self.s = [[None, None] for _ in range(2)]   # by row tile and half
        self.o = [None, None]
        self.queue = [[], []]

    def n(self, i):
        return self.items[i][0], self.items[i][1] or 0

    def at(self, i):
        """Before item i: key tiles, items and items with key tiles of each row tile, units."""
        done = self.items[:i]
        rt = [[x for x in done], [x for x in done if x[1] is not None]]
        return ([sum(x[t] for x in rt[t]) for t in range(2)], [len(rt[t]) for t in range(2)],
                [sum(x[t] > 0 for x in rt[t]) for t in range(2)], self.PER * sum(self.all[:i]))

    def long_wait(self, bar, phase):
        while not bar.ready(phase & 1):
            yield lambda: bar.ready(phase & 1)

    def copier(self):
        ok, wide = True, False
        for turn in range(len(self.items) + 1):
            i = turn if ok and turn < len(self.items) else None
            slot = turn % self.SLOTS
            if turn >= self.SLOTS:
                yield from self.long_wait(self.iempty[slot], turn // self.SLOTS - 1)
            self.item[slot] = i
            self.ifull[slot].arrive()
            yield None
            if i is None:
                return
            ok = yield from self.copy(i, wide)
            wide = self.items[i][2]

    def ready(self, bar, phase):
        yield from self.wait(bar, phase)
        return bar.ready(phase & 1)

    def copy(self, i, wide):
        tiles, items, _, units = self.at(i)
        rts = 1 if self.items[i][1] is None else 2

        def written(t):
            return items[t] == 0 or (yield from self.ready(self.qfree[t], items[t] - 1))

        def queries():
            for t in range(rts):
                if not (yield from written(t)):
                    return False
                self.check(self.q[t] in (None, "free"), "queries over an output")
                self.q[t] = i
                self.qfull[t].arrive()
                yield None
            return True
        if wide:
            for t in range(2):
                if not (yield from written(t)):
                    return False
        if not self.all[i]:
            return (yield from queries())
        for u in range(units, units + self.PER * self.all[i]):
            if u == units + 3 and not (yield from queries()):
                return False
            st = u % self.NU
            if u >= self.NU and not (yield from self.ready(self.empty[st], u // self.NU - 1)):
                return False
            self.check(self.readers[st] == 0 and self.unit[st] != "out", "unit refilled while it is read")
            self.unit[st], self.readers[st] = u, 2
            self.full[st].arrive()
            yield None
        return True

    def next_item(self, turn):
        slot = turn % self.SLOTS
        yield from self.long_wait(self.ifull[slot], turn // self.SLOTS)
        i = self.item[slot]
        self.check(i in (turn, None), "another item")
        self.iempty[slot].arrive()
        yield None
        return i

    def free(self, t, u):
        def retire():
            self.readers[u % self.NU] -= 1
            self.empty[u % self.NU].arrive()
        self.queue[t].append(retire)

    def mma(self, t):
        turn = 0
        while (i := (yield from self.next_item(turn))) is not None:
            turn += 1
            yield from self.products(t, i)
        self.queue[t].append(self.done.arrive)
        yield from self.drain(self.done)

    def products(self, t, i):
        (j0, j1), items, _, u0 = self.at(i)
        n, own = self.n(i)[t], (j0, j1)[t]
        n0 = self.n(i)[0] if self.items[i][1] is not None else 0

        def qk(j):
            if t == 1 and j < n0:
                yield from self.wait(self.sfull[0], j0 + j)
            if t == 0 and (n0 > 0 if j else j1 > 0):
                yield from self.wait(self.sfull[1], j1 + j - 1)
            for ch in range(3):
                u = u0 + self.PER * j + ch
                yield from self.wait(self.full[u % self.NU], u // self.NU)

                def retire(u=u, ch=ch):
                    self.check(self.unit[u % self.NU] == u, "S of another unit")
                    self.check(self.q[t] == i, "S of other queries")
                    self.check(ch or self.s[t] == [None, None], "S over unread weights")
                self.queue[t].append(retire)
                self.free(t, u)

            def ready():
                self.s[t] = [("S", i, j), ("S", i, j)]
                self.sfull[t].arrive()
            self.queue[t].append(ready)
        if n:
            yield from self.wait(self.qfull[t], items[t])
            yield from qk(0)
        for j in range(n):
            for h in range(2):
                u = u0 + self.PER * j + 3 + h
                yield from self.wait(self.full[u % self.NU], u // self.NU)
            yield from self.wait(self.pready[t], own + j)
            for h in range(2):
                def retire(u=u0 + self.PER * j + 3 + h, h=h, j=j):
                    self.check(self.unit[u % self.NU] == u, "O of another unit")
                    self.check(self.s[t] == [("P", i, j), ("P", i, j)], "O before its weights")
                    self.check(self.o[t] == (None if j == 0 and h == 0 else (i, j - (h == 0))), "O of another item")
                    self.o[t] = (i, j)
                    if h:
                        self.s[t] = [None, None]
                self.queue[t].append(retire)
                self.free(t, u0 + self.PER * j + 3 + h)
            yield None
            if j + 1 < n:
                yield from qk(j + 1)
        if n:
            self.queue[t].append(self.odone[t].arrive)
        for u in range(u0 + self.PER * n, u0 + self.PER * self.all[i]):
            yield from self.wait(self.full[u % self.NU], u // self.NU)
            self.free(t, u)
            yield None

    def softmax(self, t, x):
        turn = 0
        while (i := (yield from self.next_item(turn))) is not None:
            turn += 1
            if t == 0 or self.items[i][1] is not None:
                yield from self.rows(t, x, i)

    def rows(self, t, x, i):
        tiles, items, some, units = self.at(i)
        n = self.n(i)
        for j in range(n[t]):
            yield from self.wait(self.sfull[t], tiles[t] + j)
            self.check(self.s[t][x] == ("S", i, j), "S read before it is there")
            if j == 0 or self.agree:
                yield from self.meet((t, i, j), 2)
                self.check(self.o[t] == ((i, j - 1) if j else None), "O rescaled under a product")
            self.s[t][x] = ("P", i, j)
            self.pready[t].arrive()
            yield None
        yield from self.meet((t, i, "sum"), 2)
        wide = self.items[i][2]
        for r in (t, 1 - t) if wide and self.items[i][1] is not None else (t,):
            yield from self.wait(self.qfull[r], items[r])
            if n[r]:
                yield from self.wait(self.odone[r], some[r])
        if wide and self.items[i][1] is None and items[1]:
            yield from self.wait(self.qfree[1], items[1] - 1)
        self.check(n[t] == 0 or self.o[t] == (i, n[t] - 1), "output before the last product")
        self.check(self.q[t] in (i, ("out", i)), "output over other queries")
        if wide:
            end = units + self.PER * self.all[i]   # (row tile 1's reaches into the ring)
            self.check(t == 0 or all(u is None or u < end for u in self.unit), "output over units of the next item")
            self.check(self.q[1 - t] in (None, "free", i, ("out", i)), "output over another")
        self.q[t] = ("out", i)
        yield from self.meet((t, i, "out"), 2)
        yield None
        self.check(self.q[t] == ("out", i), "the output is gone")
        yield from self.meet((t, i, "read"), 2)   # (in the kernel the barrier itself counts the warps)
        self.q[t], self.o[t] = "free", None
        self.qfree[t].arrive()

    def run(self, seed, expire=None):
        self.start(seed, expire)
        self.agree = seed % 2 == 0   # with a running maximum
        self.play([self.copier()] + [self.mma(t) for t in range(2)] + [self.softmax(t, x) for t in range(2) for x in range(2)])


ITEMS = [[(2, 3, False), (1, None, True), (1, 1, False)], [(0, None, False)], [(0, 1, False)], [(1, 1, True)], [(4, 5, False), (2, 3, False), (9, 9, True), (3, None, True)],
         [(2, None, False), (1, None, False), (0, 2, False), (0, 0, False), (1, 2, False), (3, 3, False)],
         [(1, 1, False)] * 7, [(2, 2, True), (0, 1, True), (2, 2, False), (0, 3, False), (0, 3, False), (2, 2, False)]]


@pytest.mark.parametrize("items", ITEMS)
def test_prefill_random_schedules(items):
    for seed in range(60):
        Prefill(items).run(seed)


@pytest.mark.parametrize("items", ITEMS[3:])
def test_prefill_an_expired_wait_ends_every_role(items):
    for seed in range(80):
        Prefill(items).run(seed, expire=seed % 40)


@pytest.mark.parametrize("method", ["empty", "pready", "full", "qfree", "qfull", "odone"])
def test_prefill_the_model_catches_a_missing_wait(method):
    class Broken(Prefill):
        def wait(self, bar, phase):
            if bar not in getattr(self, method):
                yield from super().wait(bar, phase)

        def ready(self, bar, phase):
            yield from self.wait(bar, phase)
            return True

    with pytest.raises(AssertionError):
        for seed in range(150):
            Broken([(4, 5, False), (2, 3, False), (2, 2, True), (3, 3, False)]).run(seed)
