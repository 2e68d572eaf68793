"""How the norms' gradient exchanges a row's sums between the CTAs of a cluster, on the host: a model of its two mbarriers a
CTA under random orders of everything that may happen in another order, with a warp that gives up waiting at any call; and
the scope of that wait, which no run shows.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_matrix_10_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_sums_are_waited_for_at_cluster_scope():
    """They are stored by other CTAs, which a wait at a CTA's scope does not order before the reads."""
    waits = re.findall(r"wait_parity_bounded\(([^;]*);", source("sandwich_backward.cu"))
    assert waits and all("SharedOfCluster()" in w for w in waits)
    ptx = source("ptx.cuh")
    wait = ptx[ptx.index("int *status, SharedOfCluster) {"):]
    tries = set(re.findall(r"(mbar_try_wait\w*)\(", wait[:wait.index("return true;\n}")]))
    assert len(tries) == 1
    start = ptx.index("bool %s(" % tries.pop())
    asked = ptx[start:ptx.index("return ok", start)]
    assert ".acquire.cluster." in asked or asked.index(".relaxed.cluster.") < asked.index("fence.acquire.sync_restrict::shared::cluster.cluster")


class Broken(Exception):
    pass


class Barrier:
    """An mbarrier of one arrival a phase: the phase ends when that has come and every byte that it announced."""

    def __init__(self):
        self.phase, self.pending, self.bytes = 0, 1, 0

    def end_of_phase(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase, self.pending = self.phase + 1, 1

    def arrive_expect(self, n):
        if self.pending == 0:
            raise Broken("a second arrival in a phase")
        self.pending -= 1
        self.bytes += n
        self.end_of_phase()

    def complete(self, n):
        self.bytes -= n
        self.end_of_phase()


class Cluster:
    """ctas x warps, each through `calls` exchanges. give_up: {(cta, warp): call} of warps whose wait runs out there; after
    one has, the others' waits run out wherever nothing else can happen."""

    def __init__(self, ctas, warps, calls, rng, give_up=(), turns=2, goes_on=False, announced=None):
        self.ctas, self.warps, self.calls, self.rng, self.turns = ctas, warps, calls, rng, turns
        self.give_up, self.goes_on = dict(give_up), goes_on
        self.announced = ctas * warps * 16 if announced is None else announced
        self.bars = [[Barrier() for _ in range(turns)] for _ in range(ctas)]
        self.red = [[{} for _ in range(turns)] for _ in range(ctas)]
        self.at = {(c, w): (0, "send") for c in range(ctas) for w in range(warps)}   # (call, what comes next)
        self.flying = []     # stores under way: (to, turn, (cta, warp), call)
        self.timed_out = set()

    def ready(self, who):
        call, _ = self.at[who]
        return self.bars[who[0]][call % self.turns].phase > call // self.turns

    def runs_out(self, who, call):
        at = self.give_up.get(who, self.calls)
        return call >= at if self.goes_on else call == at

    def step(self):
        """One of the things that can happen next; False if there is none."""
        can = [("store", i) for i in range(len(self.flying))]
        for who, (call, what) in self.at.items():
            if what == "send" or (what == "wait" and (self.ready(who) or self.runs_out(who, call))):
                can.append((what, who))
        if not can:
            return False
        what, who = self.rng.choice(can)
        if what == "store":
            to, turn, sender, call = self.flying.pop(who)
            self.red[to][turn][sender] = call
            self.bars[to][turn].complete(16)
            return True
        (cta, warp), call = who, self.at[who][0]
        turn = call % self.turns
        if what == "send":
            if warp == 0:
                self.bars[cta][turn].arrive_expect(self.announced)
            self.flying += [(to, turn, who, call) for to in range(self.ctas)]
            self.at[who] = (call, "wait")
            return True
        phase = self.bars[cta][turn].phase - call // self.turns
        if phase > 1:
            raise Broken("a phase behind: its parity says that it has not ended")
        if phase < 1 or self.runs_out(who, call):
            self.leave(who)
            return True
        if any(self.red[cta][turn].get(s) != call for s in self.at):
            raise Broken("sums of another call")
        self.at[who] = (call + 1, "send" if call + 1 < self.calls else "end")
        return True

    def leave(self, who):
        self.timed_out.add(who)
        call = self.at[who][0]
        self.at[who] = (call + 1, "send") if self.goes_on and call + 1 < self.calls else (call, "end")

    def run(self):
        while True:
            if self.step():
                continue
            waiting = [who for who, (_, what) in self.at.items() if what == "wait"]
            if not waiting:
                break
            if not self.timed_out:
                raise Broken("nothing can happen any more")
            self.leave(self.rng.choice(waiting))
        assert all(what == "end" for _, what in self.at.values()) and not self.flying   # all meet at the cluster's barrier


SHAPES = [(2, 1), (2, 4), (4, 2), (8, 4)]


@pytest.mark.parametrize("ctas,warps", SHAPES)
def test_every_order_of_the_exchange_gives_the_calls_own_sums(ctas, warps):
    for seed in range(30):
        c = Cluster(ctas, warps, 7, random.Random(seed))
        c.run()
        assert not c.timed_out


@pytest.mark.parametrize("ctas,warps", SHAPES)
def test_a_wait_that_runs_out_breaks_no_barrier_and_keeps_no_warp(ctas, warps):
    for seed in range(60):
        rng = random.Random(1000 + seed)
        late = {(rng.randrange(ctas), rng.randrange(warps)): rng.randrange(7) for _ in range(rng.choice([1, 1, 2, 3]))}
        Cluster(ctas, warps, 7, rng, late).run()


@pytest.mark.parametrize("fault", [dict(turns=1), dict(announced=16), dict(announced=4096)])
def test_the_model_sees_a_faulty_exchange(fault):
    with pytest.raises(Broken):
        for seed in range(200):
            Cluster(4, 2, 7, random.Random(seed), **fault).run()


def test_the_model_sees_a_warp_that_goes_on_after_its_wait_ran_out():
    """Its next arrival may be the second in a phase, which an mbarrier of one arrival answers with a fault."""
    seen = set()
    for seed in range(200):
        try:
            Cluster(4, 2, 7, random.Random(seed), {(1, 0): 1}, goes_on=True).run()
        except Broken as e:
            seen.add(str(e))
    assert "a second arrival in a phase" in seen
