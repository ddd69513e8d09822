"""The exchange of row sums between the CTAs of a cluster (norm_fwd.cuh,
norm_bwd.cuh) when a bounded wait gives up, as a model on the CPU.

Each CTA has two mbarriers, sent[0] and sent[1], one arrival each; batch b uses
sent[b & 1].  In a batch every warp waits for the rows (`full`), warp 0 arrives
on sent[b & 1] with the bytes that are to come, every warp sends its sums to
every CTA, waits for the phase, and reads all sums.  The forward kernel has no
other barrier in a batch, the backward kernel a CTA barrier at its end.  After
the batches comes the cluster barrier, and what was sent lands at any later time.

Schedules are drawn at random, and so are the places where a wait gives up.
Whatever they are:
  * no arrival on a phase that has had its arrival,
  * no sums that overwrite some still to be read,
  * no sums that land in a CTA that has ended.
So a thread whose wait gave up arrives and sends no more, and takes part only in
the barriers.
"""
import random

import pytest


class Unsafe(Exception):
    pass


class Cta:
    def __init__(self, warps):
        self.phase, self.pending, self.bytes = [0, 0], [1, 1], [0, 0]
        self.read = [set(), set()]          # warps that still have to read the sums of the stage's last phase
        self.lost = [False] * warps         # warps that gave up: what they read does not matter
        self.at_barrier = set()             # (warp, batch)
        self.in_cluster_barrier, self.ended = 0, False

    def close(self, s):
        if self.pending[s] == 0 and self.bytes[s] == 0:
            self.phase[s], self.pending[s] = self.phase[s] + 1, 1
            return True
        return False


class Cluster:
    def __init__(self, rng, ctas, warps, batches, barrier, careful, faults):
        self.rng, self.warps, self.batches, self.barrier, self.careful = rng, warps, batches, barrier, careful
        self.cta = [Cta(warps) for _ in range(ctas)]
        self.flying = []                    # (CTA, batch) of one warp's sums
        # waits that give up although what they wait for would come
        self.faults = {(rng.randrange(ctas), rng.randrange(warps), rng.randrange(batches), rng.choice(("full", "sent")))
                       for _ in range(faults)}
        self.runs = [self.warp(c, w) for c in range(ctas) for w in range(warps)]

    def done(self, c, b):
        """Whether batch b's phase of its barrier has completed."""
        return self.cta[c].phase[b & 1] > b >> 1

    def warp(self, c, w):
        """The steps of a warp; yields where others may run.  yield f: blocked until f()."""
        me, dead = self.cta[c], -1
        for b in range(self.batches):
            if dead < 0 and (c, w, b, "full") in self.faults:
                dead = b
            yield
            if dead < 0 or not self.careful:
                if w == 0:
                    if me.pending[b & 1] == 0:
                        raise Unsafe("second arrival on a phase")
                    me.pending[b & 1] -= 1
                    me.bytes[b & 1] += len(self.cta) * self.warps
                    self.closed(c, b & 1)
                    yield
                for to in range(len(self.cta)):
                    self.flying.append((to, b))
                yield
            if dead < 0:
                tries = []
                gave_up = (c, w, b, "sent") in self.faults
                if not gave_up:
                    yield lambda: self.done(c, b) or tries.append(1) or self.stuck(tries)
                    gave_up = not self.done(c, b)
                if gave_up:
                    dead = b
            yield
            if dead < 0:
                me.read[b & 1].discard(w)  # reads the sums
            else:
                me.read = [r - {w} for r in me.read]  # its results are lost
            me.lost[w] |= dead >= 0
            yield
            if self.barrier:
                me.at_barrier.add((w, b))
                yield lambda: all((v, b) in me.at_barrier for v in range(self.warps))
        me.in_cluster_barrier += 1
        yield lambda: all(k.in_cluster_barrier == self.warps for k in self.cta)
        if w == 0:
            if self.careful and dead >= 0:
                # both phases complete, or the waits' limit passes, in which all that was sent arrives
                yield lambda: self.done(c, dead) and self.done(c, dead + 1) or not any(to == c for to, _ in self.flying)
            me.ended = True

    def stuck(self, tries):
        """A wait runs out once nothing else has moved for long."""
        return self.idle > 50 and len(tries) > 5

    def closed(self, c, s):
        if self.cta[c].close(s):
            self.cta[c].read[s] = {w for w in range(self.warps) if not self.cta[c].lost[w]}

    def land(self):
        to, b = self.flying.pop(self.rng.randrange(len(self.flying)))
        cta = self.cta[to]
        if cta.ended:
            raise Unsafe("sums land in a CTA that has ended")
        if cta.phase[b & 1] > b >> 1 or cta.phase[b & 1] < b >> 1 or cta.read[b & 1]:
            raise Unsafe("sums out of turn")
        cta.bytes[b & 1] -= 1
        self.closed(to, b & 1)

    def run(self):
        blocked = {i: None for i in range(len(self.runs))}
        self.idle = 0
        for _ in range(100000):
            if not blocked and not self.flying:
                return
            if self.flying and (not blocked or self.rng.random() < 0.3):
                self.land()
                self.idle = 0
                continue
            i = self.rng.choice(sorted(blocked))
            if blocked[i] is not None and not blocked[i]():
                self.idle += 1
                continue
            self.idle = 0
            try:
                blocked[i] = next(self.runs[i])
            except StopIteration:
                del blocked[i]
        raise AssertionError("a warp waits for good")


def trial(seed, barrier, careful, faults):
    rng = random.Random(seed)
    Cluster(rng, rng.choice((2, 3)), rng.choice((1, 2, 3)), rng.choice((1, 2, 5)), barrier, careful, faults).run()


@pytest.mark.parametrize("barrier", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("faults", [0, 1, 2])
def test_a_wait_that_gives_up_leaves_nothing_behind(barrier, faults):
    for seed in range(400):
        trial(seed, barrier, True, faults)


@pytest.mark.parametrize("barrier", [False, True], ids=["forward", "backward"])
def test_sending_on_after_a_wait_that_gave_up_is_unsafe(barrier):
    found = set()
    for seed in range(400):
        try:
            trial(seed, barrier, False, 1)
        except Unsafe as e:
            found.add(str(e))
    assert found == {"second arrival on a phase", "sums out of turn", "sums land in a CTA that has ended"}
