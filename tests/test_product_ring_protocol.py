"""The rings of the int8 product (gemm_i8_kernel) and of the gradient products
(gemm_grad_kernel), simulated on the CPU, with their bounded waits and the way out
when one runs out.

A cluster of two CTAs computes a tile.  Per stage each CTA's TMA thread loads its
halves of both operands; all bytes count on the leader CTA's "full" barrier, which
also takes one arrival, the leader's own (the peer's bytes may land before it).  The
leader's MMA thread takes the stages in order; when the MMAs of a stage complete they
arrive on the stage's "empty" barrier in both CTAs.  A run of stages accumulates in
one of two halves of tensor memory; its completion arrives on "accumulator full" in
both CTAs, whose epilogue warps read it and arrive (remotely) on the leader's
"accumulator empty".  The int8 product's run is its tile's whole contraction; the
gradient products' is at most 4 or 8 stages.

Each wait ends: when its barrier completes, when another role of the same CTA has
given up (not the waits that drain), or when its limit runs out.  The simulation runs
random interleavings, with copies and MMAs that complete later, and reports reads of
a stage or accumulator that does not hold what the reader wants, writes over what is
still to be read, and, after the teardown that both CTAs enter together, copies or
MMAs still in flight.  Failures: a TMA thread that stops, copies that never land.
"""
import random

import pytest

WARPS = 4       # epilogue warps per CTA (the kernels have 16 and 8: no difference to the protocol)


class Barrier:
    """mbarrier: arrivals and bytes of a phase."""

    def __init__(self, count):
        self.count = self.pending = count
        self.bytes = 0
        self.completed = 0

    def _check(self):
        assert self.pending >= 0
        if self.pending == 0 and self.bytes == 0:
            self.completed += 1
            self.pending = self.count

    def arrive(self, expect=0):
        self.bytes += expect
        self.pending -= 1
        self._check()

    def landed(self, n):
        self.bytes -= n
        self._check()

    def try_wait_parity(self, parity):
        return (self.completed + 1) % 2 == parity


class Cluster:
    def __init__(self, stages, runs, seed, limit=10 ** 9, stop=None, lost=None, skip_acce=False, skip_drain=False):
        self.S, self.runs, self.limit = stages, runs, limit
        self.stop, self.lost, self.skip_acce, self.skip_drain = stop, lost, skip_acce, skip_drain
        self.rng = random.Random(seed)
        self.now, self.bad, self.flags = 0, [], set()
        self.full = [Barrier(1) for _ in range(stages)]                          # leader
        self.empty = [[Barrier(1) for _ in range(stages)] for _ in range(2)]     # both CTAs
        self.accf = [[Barrier(1) for _ in range(2)] for _ in range(2)]           # both CTAs
        self.acce = [Barrier(2 * WARPS) for _ in range(2)]                       # leader
        self.drain = Barrier(1)                                                  # leader
        self.abort = [False, False]
        self.holds = [[None] * stages for _ in range(2)]
        self.done_mmas, self.readers = set(), {}
        self.acc = [None, None]
        self.events = []            # (time, function)
        self.copies = self.mmas = 0
        self.mma_clock = 0          # MMAs and commits complete in order

    def later(self, lo, hi, f):
        self.events.append((self.now + self.rng.randint(lo, hi), f))

    def wait(self, bar, parity, cta, drain=False):
        t0 = self.now
        while not bar.try_wait_parity(parity):
            if (not drain and self.abort[cta]) or self.now - t0 > self.limit:
                return False
            yield
        return True

    def fail(self, cta, site):
        self.flags.add(site)
        self.abort[cta] = True

    def producer(self, c):
        total, it = sum(self.runs), 0
        while it < total:
            s = it % self.S
            if self.stop is not None and self.stop[0] == c and it >= self.stop[1]:
                break
            if not (yield from self.wait(self.empty[c][s], ((it // self.S) & 1) ^ 1, c)):
                self.fail(c, "producer")
                break
            if it >= self.S and it - self.S not in self.done_mmas:
                self.bad.append(("overwrite", c, it))
            if c == 0:
                self.full[s].arrive(expect=4)
            for part in range(2):           # two copies, one byte each
                self.copies += 1

                def land(it=it, s=s, part=part):
                    self.copies -= 1
                    if part == 1:
                        self.holds[c][s] = it
                    self.full[s].landed(1)
                if self.lost != (c, it):
                    self.later(1, 8, land)
                else:
                    self.copies -= 1
            it += 1
            yield
        if self.skip_drain:
            return
        for j in range(max(0, it - self.S), it):
            if not (yield from self.wait(self.empty[c][j % self.S], (j // self.S) & 1, c, drain=True)):
                break

    def commit(self, f):
        self.mma_clock = max(self.mma_clock + 1, self.now + self.rng.randint(1, 10))
        self.mmas += 1

        def complete():
            self.mmas -= 1
            f()
        self.events.append((self.mma_clock, complete))

    def issuer(self):
        it, ok = 0, True
        for n, length in enumerate(self.runs):
            a = n & 1
            if not self.skip_acce and not (yield from self.wait(self.acce[a], ((n >> 1) & 1) ^ 1, 0)):
                self.fail(0, "accumulator")
                break
            if n >= 2 and self.readers.get(n - 2, 0) != 2 * WARPS:
                self.bad.append(("accumulator overwritten", n))
            self.acc[a] = ("partial", n)
            for _ in range(length):
                s = it % self.S
                if not (yield from self.wait(self.full[s], (it // self.S) & 1, 0)):
                    self.fail(0, "stage")
                    ok = False
                    break
                if any(self.holds[c][s] != it for c in range(2)):
                    self.bad.append(("early read", it))

                def stage_done(it=it, s=s):
                    self.done_mmas.add(it)
                    for c in range(2):
                        self.empty[c][s].arrive()
                self.commit(stage_done)
                it += 1
                yield
            if not ok:
                break

            def run_done(n=n, a=a):
                self.acc[a] = ("whole", n)
                for c in range(2):
                    self.accf[c][a].arrive()
            self.commit(run_done)
        self.commit(self.drain.arrive)
        yield from self.wait(self.drain, 0, 0, drain=True)

    def epilogue(self, c):
        for n in range(len(self.runs)):
            a = n & 1
            if not (yield from self.wait(self.accf[c][a], (n >> 1) & 1, c)):
                self.fail(c, "epilogue")
                return
            if self.acc[a] != ("whole", n):
                self.bad.append(("early accumulator", c, n, self.acc[a]))
            for _ in range(self.rng.randint(0, 4)):
                yield
            self.readers[n] = self.readers.get(n, 0) + 1
            self.acce[a].arrive()
            yield

    def run(self, most=200000):
        """Steps until every role of both CTAs has ended; None if that takes too long."""
        roles = [self.producer(0), self.producer(1), self.issuer()] + [self.epilogue(c) for c in range(2)
                                                                        for _ in range(WARPS)]
        while roles and self.now < most:
            self.now += 1
            for e in [e for e in self.events if e[0] <= self.now]:
                self.events.remove(e)
                e[1]()
            self.rng.shuffle(roles)
            for r in list(roles):
                if self.rng.random() < 0.7:
                    try:
                        next(r)
                    except StopIteration:
                        roles.remove(r)
        if roles:
            return None
        if self.copies or self.mmas:
            self.bad.append(("in flight at the teardown", self.copies, self.mmas))
        return self.now


def cut(stages, most):
    return [most] * (stages // most) + ([stages % most] if stages % most else [])


# (stages of the ring, runs): int8, several tiles; dx with its long and short ring; dW with both (a unit's last run may
# be shorter), and runs shorter than the ring is deep
FORMS = [(5, [25] * 4), (5, [1] * 9), (5, [3, 4, 3, 4]), (6, cut(52, 8) * 2), (5, cut(9, 8) * 4), (4, cut(34, 4) * 2),
         (3, cut(5, 4) * 6)]


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("seed", range(6))
def test_every_stage_and_accumulator_is_read_in_time(form, seed):
    c = Cluster(*FORMS[form], seed=seed)
    assert c.run() is not None
    assert c.bad == [] and not c.flags
    assert all(c.readers[n] == 2 * WARPS for n in range(len(c.runs)))


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("stop", [(0, 0), (1, 0), (0, 3), (1, 4), "lost 0", "lost 1", "both"])
def test_a_wait_that_runs_out_ends_every_role(form, stop):
    """A TMA thread that stops (from the start, as the self test has it, or later), or a copy that never lands: each
    role ends within a few limits, the failure is flagged, and nothing that was issued is still on its way (the lost copy
    apart)."""
    limit = 300
    for seed in range(4):
        kw = dict(lost=(int(stop[-1]), 2)) if isinstance(stop, str) and stop != "both" else {}
        c = Cluster(*FORMS[form], seed=seed, limit=limit, stop=stop if isinstance(stop, tuple) else None, **kw)
        if stop == "both":
            c.producer = lambda cta: iter(())
        end = c.run()
        assert end is not None and end < 6 * limit, end
        assert c.flags and c.bad == []


def test_simulation_sees_planted_mistakes():
    hits = [b[0] for seed in range(10) for c in [Cluster(5, [2] * 12, seed, skip_acce=True)] if c.run() for b in c.bad]
    assert "accumulator overwritten" in hits or "early accumulator" in hits
    # a TMA thread that leaves without draining, while the other has stopped
    hits = []
    for seed in range(10):
        c = Cluster(5, [25], seed, limit=1, stop=(0, 2), skip_drain=True)
        c.run()
        hits += [b[0] for b in c.bad]
    assert "in flight at the teardown" in hits
