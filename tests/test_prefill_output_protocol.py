"""Model of the queries' and the output's use of shared memory in the prefill
kernel (csrc/pa_prefill_umma.cuh), under random schedules on the CPU.

Every softmax warp stores a share of the queries of every row tile and arrives
on `qfull`, for which the MMA warps wait.  At its end a warp writes its part
of the output over the queries (a bf16 tile over its own, fp32 rows of tile 0
over both tiles'), meets the other half's warp of its pair and reads it back.
One pair per row tile runs in full; the warps of another pair, which it never
meets, store their queries at times of their own.  A query
stored between the write and the read would reach the output; a query
overwritten before its products read it would spoil them.  A tile whose rows
see no key has no products, so nothing but `qfull` orders the two."""
import pytest

from tests.test_prefill_protocol import FORMS, Prefill
from tests.test_verify_protocol import Bar


class Output(Prefill):
    def __init__(self, form, tiles, quant, wide, **kw):
        super().__init__(form, tiles, quant, **kw)
        self.wide, self.warps = wide, 4 * self.RT
        self.qfull = Bar(self.warps)
        self.stored = [0] * self.RT          # warps whose queries of a row tile are there
        self.written = [set() for _ in range(self.RT)]   # warps whose output lies over them
        for _ in range(2 * self.RT):         # the warps of the other pairs
            self.queue.append([lambda r=r: self.store(r) for r in range(self.RT)] + [self.qfull.arrive])

    def store(self, r):
        self.check(not self.written[r], "query stored over an output")
        self.stored[r] += 1

    def ends_wait_for_queries(self):
        return self.n == 0

    def mma(self, t):
        yield from self.wait(self.qfull, 0)
        yield from super().mma(t)
        while any(self.queue[self.RT:]):     # every warp of the CTA meets the others at its end
            yield lambda: not any(self.queue[self.RT:])

    def qk(self, t, u, j, h, buf, halves):
        super().qk(t, u, j, h, buf, halves)
        product = self.queue[t].pop()

        def retire():
            self.check(self.stored[t] == self.warps, "product of queries that are not there")
            self.check(not self.written[t], "product of overwritten queries")
            product()
        self.queue[t].append(retire)

    def softmax(self, t, x, rng):
        for r in range(self.RT):
            self.store(r)
            yield None
        self.qfull.arrive()
        yield from super().softmax(t, x, rng)
        if self.ends_wait_for_queries():
            yield from self.wait(self.qfull, 0)
        # fp32 rows of tile 1 lie past the queries, over units that are all used
        over = range(self.RT) if self.wide and t == 0 else [] if self.wide else [t]
        for r in over:
            self.written[r].add((t, x))
        yield from self.meet((t, "output"))
        for r in over:
            self.check(self.stored[r] == self.warps, "output read back before the last query was stored")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n", [0, 1, 2, 5])
def test_random_schedules(form, n, wide):
    for seed in range(60):
        Output(form, n, form == "d256", wide).run(seed)


@pytest.mark.parametrize("form", FORMS)
def test_an_expired_wait_ends_every_role(form):
    for n in (0, 4):
        for seed in range(40):
            Output(form, n, False, True).run(seed, expire=seed % 12)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("form", FORMS)
def test_the_model_catches_an_output_that_does_not_wait_for_the_queries(form, wide):
    class Broken(Output):
        def ends_wait_for_queries(self):
            return False

    with pytest.raises(AssertionError):
        for seed in range(80):
            Broken(form, 0, False, wide).run(seed)
