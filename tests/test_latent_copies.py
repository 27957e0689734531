"""The stream of items of the expanded form (csrc/pa_latent_prefill.cu) and the run of
pieces of the absorbed one (csrc/pa_latent_rows.cu) with copies that land later than they
are issued, in any order between barriers, under random schedules on the CPU.  The models
of test_latent_protocol let them land at once; what passes a barrier a phase too early can
then not be seen."""
import random

import pytest

from tests.test_latent_protocol import ITEMS, PIECES, Prefill, Rows
from tests.test_verify_protocol import Bar


class InFlight(Prefill):
    """every: a row tile's products wait for its queries in every item that has the row
    tile, also without key tiles.  back: and hold the next ones back until then.
    both: the queries of an item with a wide output wait for what both row tiles wrote.
    stop: nothing is copied once a wait has expired (the arrivals that follow are void).
    issued: the copies waited for at the end are those that were issued, not all of the
    items that were begun."""

    def __init__(self, items, every=True, back=True, both=True, stop=True, issued=True):
        super().__init__(items)
        self.every, self.back, self.both, self.stop, self.issued = every, back, both, stop, issued
        self.sent, self.units, self.begun = [0, 0], 0, 0
        if back:
            self.qfree = [Bar(3) for _ in range(2)]
        self.queue += [[] for _ in range(2 + self.NU)]   # copies on their way, by barrier

    def land(self, q, f):
        self.queue[2 + q] += [lambda: None] * self.rng.choice((0, 1, 20)) + [f]

    def ready(self, bar, phase):
        ok = yield from super().ready(bar, phase)
        return ok and not (self.stop and self.abort)

    def copier(self):
        yield from super().copier()
        sent, units = self.sent, self.units
        if not self.issued:
            _, sent, _, units = self.at(self.begun)
        for t in range(2):
            if sent[t]:
                yield from self.long_wait(self.qfull[t], sent[t] - 1)
        for u in range(max(0, units - self.NU), units):
            yield from self.long_wait(self.full[u % self.NU], u // self.NU)
        assert not any(self.queue[2:]), "copies in flight at the end"

    def copy(self, i, wide):
        self.begun = i + 1
        tiles, items, _, units = self.at(i)
        rts = 1 if self.items[i][1] is None else 2

        def written(t):
            return items[t] == 0 or (yield from self.ready(self.qfree[t], items[t] - 1))

        def queries():
            if self.both and self.items[i][2] and not (yield from written(1)):
                return False
            for t in range(rts):
                if not (yield from written(t)):
                    return False
                self.check(self.q[t] in (None, "free"), "queries over an output")
                self.q[t] = ("on its way", i)

                def there(t=t):
                    self.check(self.q[t] == ("on its way", i), "queries over something else")
                    self.q[t] = i
                    self.qfull[t].arrive()
                self.land(t, there)
                self.sent[t] += 1
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
            self.check(self.readers[st] == 0, "unit refilled while it is read")
            self.unit[st], self.readers[st] = u + 0.5, 2   # (on its way: no whole number)

            def there(u=u):
                self.unit[u % self.NU] = u
                self.full[u % self.NU].arrive()
            self.land(2 + st, there)
            self.units += 1
            yield None
        return True

    def products(self, t, i):
        if t == 0 or self.items[i][1] is not None:
            if self.every:
                yield from self.wait(self.qfull[t], self.at(i)[1][t])
            if self.back:
                self.qfree[t].arrive()
                yield None
        yield from super().products(t, i)

    def rows(self, t, x, i):
        tiles, items, some, units = self.at(i)
        n, (_, second, wide) = self.n(i), self.items[i]
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
        yield from self.wait(self.qfull[t], items[t])
        if n[t]:
            yield from self.wait(self.odone[t], some[t])
        if wide and second is None and items[1] and not self.both:
            yield from self.wait(self.qfree[1], items[1] - 1)
        if wide and second is not None:
            yield from self.wait(self.qfull[1 - t], items[1 - t])
            if n[1 - t]:
                yield from self.wait(self.odone[1 - t], some[1 - t])
        self.check(n[t] == 0 or self.o[t] == (i, n[t] - 1), "output before the last product")
        self.check(self.q[t] in (i, ("out", i)), "output over other queries")
        if wide:
            end = units + self.PER * self.all[i]   # (row tile 1's reaches into the ring)
            self.check(t == 0 or all(u is None or u < end for u in self.unit), "output over units of the next item")
            self.check(self.q[1 - t] in (None, "free", i, ("out", i)), "output over another")
            self.check(second is None or self.o[1 - t] in (None, (i, n[1 - t] - 1)), "output over queries in use")
        self.q[t] = ("out", i)
        yield from self.meet((t, i, "out"), 2)
        yield None
        self.check(self.q[t] == ("out", i), "the output is gone")
        yield from self.meet((t, i, "read"), 2)   # (in the kernel the barrier itself counts the warps)
        self.q[t], self.o[t] = "free", None
        self.qfree[t].arrive()


STREAMS = ITEMS + [[(0, 0, True), (2, 2, False)], [(0, 0, False), (1, 2, False), (0, 0, False), (0, 0, False), (2, 2, False)],
                   [(1, 1, False)] + [(0, 0, False)] * 6 + [(0, None, False)] * 5 + [(1, 2, False)],
                   [(0, None, True), (3, None, True), (0, 0, True), (0, 1, True), (2, 2, True)],
                   [(1, 1, False), (0, 1, True)], [(3, None, False), (1, 1, True), (0, 0, False), (0, 0, True)],
                   [(2, 2, False), (0, 1, True), (1, 1, False), (1, 1, True), (0, None, True)]]


@pytest.mark.parametrize("items", STREAMS)
def test_copies_that_land_late(items):
    for seed in range(60):
        InFlight(items).run(seed)


def some_items(rng):
    """Row tile 1 sees as many key tiles as row tile 0, or one more; wide or not, or mixed."""
    wide, items = rng.choice((False, True, None)), []
    for _ in range(rng.randint(2, 9)):
        n = rng.choice((0, 0, 1, 2, 3))
        items.append((n, rng.choice((None, n, n + 1)), rng.random() < 0.4 if wide is None else wide))
    return items


@pytest.mark.parametrize("seed", range(40))
def test_any_stream(seed):
    items = some_items(random.Random(seed))
    for k in range(20):
        InFlight(items).run(k)
        InFlight(items).run(k, expire=3 * k)


@pytest.mark.parametrize("items", STREAMS)
def test_an_expired_wait_leaves_no_copy_in_flight(items):
    for seed in range(60):
        InFlight(items).run(seed, expire=seed % 30)


def test_copies_must_end_with_an_expired_wait():
    with pytest.raises(AssertionError, match="in flight"):
        for seed in range(200):
            InFlight([(4, 5, False), (2, 3, False), (2, 2, False)], stop=False).run(seed, expire=seed % 30)


def test_copies_that_were_never_issued_must_not_be_waited_for():
    with pytest.raises(AssertionError, match="deadlock|in flight"):
        for seed in range(60):
            InFlight([(4, 5, False), (2, 3, False)], issued=False).run(seed, expire=seed % 30)


@pytest.mark.parametrize("items", [[(0, 0, True), (2, 2, True)], [(0, 0, False), (1, 1, False)],
                                   [(1, 1, False), (0, None, False), (1, None, False)]])
def test_a_row_tile_without_keys_must_wait_for_its_queries(items):
    """Else the next item passes on the phase of queries that are still on their way."""
    with pytest.raises(AssertionError, match="queries"):
        for seed in range(150):
            InFlight(items, every=False, back=False).run(seed)


def test_a_row_tile_without_keys_must_not_be_left_behind():
    """Else its queries' phase is over, and the next one's, before it has looked."""
    with pytest.raises(AssertionError, match="deadlock"):
        for seed in range(400):
            InFlight([(0, 0, False)] * 40, back=False).run(seed)


def test_a_wide_output_must_wait_for_both_row_tiles():
    """A narrow item, then one in pieces of which row tile 0 sees nothing."""
    with pytest.raises(AssertionError, match="output over another"):
        for seed in range(400):
            InFlight([(1, 1, False), (0, 1, True)], both=False).run(seed)


class RowsInFlight(Rows):
    """stop: nothing is copied once a wait has expired."""

    def __init__(self, pieces, safe=False, stages=4, early_q=True, stop=True):
        super().__init__(pieces, False, safe, stages, early_q)
        self.stop = stop
        self.queue += [[] for _ in range(1 + stages)]

    def land(self, q, f):
        self.queue[2 + q] += [lambda: None] * self.rng.choice((0, 1, 20)) + [f]

    def ready(self, bar, phase):
        yield from self.wait(bar, phase)
        return bar.ready(phase & 1) and not (self.stop and self.abort)

    def copier(self, which, of):
        g = 0
        for _, _, g in self.tiles():
            st = g % self.NS
            if g >= self.NS and not (yield from self.ready(self.empty[st], g // self.NS - 1)):
                break
            self.check(self.readers[st] == 0, "stage refilled while it is read")
            self.stage[st], self.readers[st] = ("on its way", g), 2

            def there(g=g):
                self.stage[g % self.NS] = g
                self.full[g % self.NS].arrive()
            self.land(1 + st, there)
            yield None
        else:
            g = sum(1 for _ in self.tiles())
        yield from self.landed([(self.full[u % self.NS], u // self.NS) for u in range(max(0, g - self.NS), g)])
        assert not any(self.queue[3:]), "tiles in flight at the end"

    def query(self):
        sent = 0
        for i in range(len(self.pieces)):
            if i and not (yield from self.ready(self.qfree, i - 1)):
                break
            self.qsmem = ("on its way", i)

            def there(i=i):
                self.qsmem = i
                self.qfull.arrive()
            self.land(0, there)
            sent += 1
            yield None
        yield from self.landed([(self.qfull, sent - 1)] if sent else [])
        assert not self.queue[2], "queries in flight at the end"

    def landed(self, last):   # no abort ends these waits
        for bar, phase in last:
            while not bar.ready(phase & 1):
                yield lambda: bar.ready(phase & 1)


@pytest.mark.parametrize("pieces", PIECES)
def test_rows_copies_that_land_late(pieces):
    for seed in range(60):
        for safe in (False, True):
            RowsInFlight(pieces, safe, 4 + seed % 2, seed % 3 > 0).run(seed)


@pytest.mark.parametrize("pieces", PIECES)
def test_rows_an_expired_wait_leaves_no_copy_in_flight(pieces):
    for seed in range(100):
        RowsInFlight(pieces, seed % 2 == 0, 4 + seed % 2, seed % 3 > 0).run(seed, expire=seed % 40)


def test_rows_copies_must_end_with_an_expired_wait():
    with pytest.raises(AssertionError, match="in flight"):
        for seed in range(200):
            RowsInFlight([3, 1, 6], stop=False).run(seed, expire=seed % 30)
