"""After an expired wait the INT8 product's CTAs wait for every copy that was asked for, whichever role gave up (CPU).

csrc/ring.h, the kernels' own arithmetic of what to wait for, is compiled for the host.  Around it the roles are played
here on barriers with the hardware's phase rule (a wait for parity P ends while the last completed phase has parity P):
loaders that refill stages as they are released, issuers that release a stage some time after its copy landed, copies
that land whenever they like, and a wait of some role that gives up at any moment, upon which every role leaves at its
next wait.
"""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_quant_b200", "csrc")


@pytest.fixture(scope="module")
def last_use(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src, so = d / "ring.cpp", d / "ring.so"
    src.write_text('#include "ring.h"\nextern "C" long long last_use(long long n, int s, int stages) '
                   '{ return ssd::ring_last_use(n, s, stages); }\n')
    subprocess.run(["g++", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(src)], check=True)
    f = ctypes.CDLL(str(so)).last_use
    f.argtypes, f.restype = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int], ctypes.c_longlong
    return f


def test_last_use_by_counting(last_use):
    for stages in range(1, 17):
        for n in range(0, 70):
            for s in range(stages):
                assert last_use(n, s, stages) == len(range(s, n, stages)) - 1
    assert last_use(2 ** 40 + 3, 2, 6) == (2 ** 40 + 3 - 1 - 2) // 6


class Barrier:
    def __init__(self):
        self.done = 0                                   # completed phases

    def passed(self, parity):
        return (self.done & 1) != parity


class Cta:
    """matmul_few_kernel's loading and issuing roles on one ring."""

    def __init__(self, rng, slices, stages, issue):
        self.rng, self.slices, self.stages, self.issue = rng, slices, stages, issue
        self.full = [Barrier() for _ in range(stages)]
        self.empty = [Barrier() for _ in range(stages)]
        self.flying, self.landed, self.mma = [], set(), []
        first = min(stages, slices)
        for j in range(first):
            self.flying.append(j)
        self.j = [first + w for w in range(issue)]      # per loading role: its next slice
        self.i = list(range(issue))                     # per issuing role
        self.abort = False
        self.gave_up = None

    def events(self):
        ev = [("land", j) for j in self.flying] + [("mma", j) for j in self.mma]
        if not self.abort:
            for w in range(self.issue):
                j = self.j[w]
                if j < self.slices and self.empty[j % self.stages].passed((j // self.stages - 1) & 1):
                    ev.append(("load", w))
                i = self.i[w]
                if i < self.slices and self.full[i % self.stages].passed((i // self.stages) & 1):
                    ev.append(("issue", w))
        return ev

    def step(self, ev):
        kind, v = ev
        if kind == "land":
            self.flying.remove(v)
            self.full[v % self.stages].done += 1
            assert self.full[v % self.stages].done == v // self.stages + 1      # copies of a stage land in order
        elif kind == "mma":
            self.mma.remove(v)
            self.empty[v % self.stages].done += 1
        elif kind == "load":
            self.flying.append(self.j[v])
            self.j[v] += self.issue
        else:
            self.mma.append(self.i[v])
            self.i[v] += self.issue

    def run_until_abort(self, moment):
        for n in range(10 ** 6):
            ev = self.events()
            if n == moment:
                self.abort = True
                waiting = [("loader", w) for w in range(self.issue) if self.j[w] < self.slices]
                waiting += [("issuer", w) for w in range(self.issue) if self.i[w] < self.slices]
                self.gave_up = self.rng.choice(waiting) if waiting else None
                return
            if not ev:
                return
            self.step(self.rng.choice(ev))


def _finish_waits(cta, waits):
    """The waits (stage, parity) one after the other; what happens meanwhile happens at random.  False: one never ends."""
    for s, parity in waits:
        while not cta.full[s].passed(parity):
            ev = [e for e in cta.events() if e[0] in ("land", "mma")]
            if not ev:
                return False
            cta.step(cta.rng.choice(ev))
    return True


SHAPES = [(slices, stages, issue) for issue in (1, 2) for slices in (1, 2, 3, 5, 8, 20, 33)
          for stages in ((2, 4, 10) if issue == 2 else (1, 3, 5)) if slices > stages or issue == 1] + \
         [(n, n, 2) for n in (1, 2, 3, 7)]


@pytest.mark.parametrize("slices,stages,issue", SHAPES)
def test_no_copy_is_left_when_a_role_gave_up(last_use, slices, stages, issue):
    stages = min(stages, slices)
    rng = random.Random(slices * 100 + stages * 10 + issue)
    old_rule_left_some = False
    for _ in range(400):
        cta = Cta(rng, slices, stages, issue)
        cta.run_until_abort(rng.randrange(1, 6 * slices + 2))
        waits = []
        for s in range(stages):
            u = last_use(min(cta.j[s % issue], slices), s, stages)
            if u >= 0:
                waits.append((s, int(u) & 1))
        assert _finish_waits(cta, waits)
        assert not cta.flying, (cta.gave_up, cta.j, cta.i)
        # the rule of waiting only in a loader whose own wait gave up, on the same schedule
        if cta.gave_up and cta.gave_up[0] == "issuer" and all(j >= slices for j in cta.j):
            old_rule_left_some = True
    assert old_rule_left_some                             # that rule has no wait at all in these


@pytest.mark.parametrize("stages", [5, 6])
def test_pair_waits_for_both_ctas_copies(last_use, stages):
    """matmul_pair_kernel: a slice's copies into both CTAs complete the even CTA's phase, whose arrival the even CTA
    gives when it asks for its own.  The waits are for the slices that either asked for."""
    rng = random.Random(stages)
    for _ in range(2000):
        total = rng.randrange(0, 40)
        ahead = rng.choice([0, 0, rng.randrange(0, stages + 1)])
        even, odd = (total, total + ahead) if rng.random() < 0.5 else (total + ahead, total)
        flying = {(c, k) for c, n in ((0, even), (1, odd)) for k in range(n) if n - k <= stages and rng.random() < 0.7}
        # a stage's earlier slice had to be complete before the stage was asked for again
        flying = {(c, k) for c, k in flying if k >= max(even, odd) - stages}

        def done(s):
            n = 0
            for k in range(s, max(even, odd), stages):
                if k >= even or k >= odd or (0, k) in flying or (1, k) in flying:
                    break
                n += 1
            return n

        open_phase = False
        for s in range(stages):
            u = last_use(max(even, odd), s, stages)
            if u < 0:
                continue
            while (done(s) & 1) == (int(u) & 1):          # the phase of parity u & 1 is not complete
                mine = [f for f in flying if f[1] % stages == s]
                if mine:
                    flying.remove(rng.choice(mine))
                else:
                    assert even != odd                    # one CTA never asked: the deadline ends the wait
                    open_phase = True
                    break
        assert not flying or open_phase
        assert not flying or even != odd
