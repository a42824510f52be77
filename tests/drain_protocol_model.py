"""Host-side models of how the tcgen05 kernels end: nothing may be in flight when a CTA releases its memory.

The warp roles of a kernel are Python generators that hand work to one another through mbarriers with the
kernel's arrival counts and phase parities. TMA copies land in any order, the commits of one issuing thread in
theirs, at times the scheduler picks. A wait can run out of time: it raises the abort flag, after which a wait
whose phase has not completed returns false and its role leaves. `late` lets that happen only once the
producers have left, while their last copies are still on their way: a producer that looks at the flag when it
leaves sees nothing then.

A run returns "ok" or "aborted"; it raises Hazard when a role uses or overwrites a buffer out of turn, when the CTA
ends with copies or products in flight, and when a wait on the way out (which ignores the flag) waits for a
phase that does not come.
"""
from __future__ import annotations

import random


class Hazard(Exception):
    pass


def check(cond, msg):
    if not cond:
        raise Hazard(msg)


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


class Sim:
    """Roles yield ("wait", barrier, parity) -> bool, ("drain", barrier, parity) or ("until", condition)."""

    def __init__(self, rng, timeout_p=0.0, late=False):
        self.rng, self.timeout_p, self.late = rng, timeout_p, late
        self.bars, self.roles, self.pending, self.abort, self.producers = {}, {}, [], False, set()

    def bar(self, name, count):
        self.bars[name] = Bar(count)

    def copy(self, issuer, fn):          # a TMA load: lands in any order
        self.pending.append(("tma " + issuer, fn))

    def commit(self, issuer, fn):        # an MMA issuer's commit: in order
        self.pending.append(("mma " + issuer, fn))

    def _value(self, want):
        kind = want[0]
        if kind == "until":
            return True if want[1]() else None
        if self.bars[want[1]].passed(want[2]):
            return True
        return False if kind == "wait" and self.abort else None

    def run(self, max_steps=200_000):
        want = {}

        def step(name, value):
            try:
                want[name] = self.roles[name].send(value)
            except StopIteration:
                want[name] = None

        for name in self.roles:
            step(name, None)
        for _ in range(max_steps):
            live = [k for k, v in want.items() if v is not None]
            if not live:
                check(not self.pending, "the CTA ends with work in flight: " + ", ".join(i for i, _ in self.pending))
                return "aborted" if self.abort else "ok"
            gone = all(want[p] is None or want[p][0] == "drain" for p in self.producers)
            if not self.abort and (gone or not self.late) and self.rng.random() < self.timeout_p:
                blocked = [k for k in live if want[k][0] == "wait" and self._value(want[k]) is None]
                if blocked:
                    self.abort = True
                    continue
            choices = [("role", k) for k in live if self._value(want[k]) is not None]
            copies = [i for i, (who, _) in enumerate(self.pending) if who.startswith("tma ")]
            if not (self.late and not gone and choices):     # late: copies land last
                choices += [("land", i) for i in copies]
            firsts = {}
            for i, (who, _) in enumerate(self.pending):
                if who.startswith("mma "):
                    firsts.setdefault(who, i)
            choices += [("land", i) for i in firsts.values()]
            if not choices:
                stuck = "; ".join(f"{k}: {want[k][0]} {want[k][1:]}" for k in live)
                if all(want[k][0] != "wait" for k in live):
                    raise Hazard("a wait on the way out waits for nothing: " + stuck)
                check(not self.abort, "stuck after the abort: " + stuck)
                self.abort = True                            # a bounded wait runs out
                continue
            kind, who = self.rng.choice(choices)
            if kind == "role":
                step(who, self._value(want[who]))
            else:
                self.pending.pop(who)[1]()
        raise Hazard("step limit")


def gemm(kblocks, stages, rng, timeout_p=0.0, late=False, drain="always", hold=False):
    """gemm_kernel<false, BN>: tiles of kblocks[n] k blocks through `stages` stages and two accumulators, with a
    producer, an MMA issuer and epilogue warps (two here). drain: "always" (the kernel), "flag" (only if the
    abort flag is up when the producer leaves) or "never". hold: the epilogue waits for a release nothing gives."""
    s = Sim(rng, timeout_p, late)
    n_ep = 2
    for i in range(stages):
        s.bar(f"FULL{i}", 1)
        s.bar(f"EMPTY{i}", 1)
    for i in range(2):
        s.bar(f"AFULL{i}", 1)
        s.bar(f"AEMPTY{i}", n_ep)
    s.bar("DRAIN", 1)
    s.bar("HOLD", 1)
    held, used, acc, stored = [None] * stages, [-1], [None, None], [0, 0]
    B = s.bars

    def producer():
        it, ok = 0, True
        for n in range(len(kblocks)):
            for _ in range(kblocks[n]):
                if not ok:
                    break
                st = it % stages
                ok = yield "wait", f"EMPTY{st}", ((it // stages) & 1) ^ 1
                if not ok:
                    break
                check(used[0] >= it - stages, "a stage is filled before its products have read it")

                def land(st=st, it=it):
                    held[st] = it
                    B[f"FULL{st}"].arrive()
                s.copy("p", land)
                it += 1
        if drain == "always" or (drain == "flag" and s.abort):
            for j in range(max(0, it - stages), it):
                yield "drain", f"FULL{j % stages}", (j // stages) & 1

    def mma():
        it, ok = 0, True
        for n in range(len(kblocks)):
            if not ok:
                break
            ab = n & 1
            ok = yield "wait", f"AEMPTY{ab}", ((n >> 1) & 1) ^ 1
            if ok:
                check(n < 2 or stored[ab] == n_ep * (n // 2), "an accumulator is overwritten before it is read")
            for _ in range(kblocks[n]):
                if not ok:
                    break
                st = it % stages
                ok = yield "wait", f"FULL{st}", (it // stages) & 1
                if not ok:
                    break
                check(held[st] == it, "a product reads a stage that holds something else")

                def done(st=st, it=it):
                    used[0] = it
                    B[f"EMPTY{st}"].arrive()
                s.commit("m", done)
                it += 1
            if ok:
                def full(ab=ab, n=n):
                    acc[ab] = n
                    B[f"AFULL{ab}"].arrive()
                s.commit("m", full)
        s.commit("m", B["DRAIN"].arrive)
        yield "drain", "DRAIN", 0

    def epilogue():
        for n in range(len(kblocks)):
            ab = n & 1
            if not (yield "wait", f"AFULL{ab}", (n >> 1) & 1):
                return
            if hold and n == 0 and not (yield "wait", "HOLD", 0):
                return
            check(acc[ab] == n, "the epilogue reads another tile's accumulator")
            stored[ab] += 1
            B[f"AEMPTY{ab}"].arrive()

    s.roles = {"producer": producer(), "mma": mma(), **{f"epilogue {i}": epilogue() for i in range(n_ep)}}
    s.producers = {"producer"}
    return s.run()


def random_gemm(rng):
    stages = rng.choice([2, 3, 6])
    return [rng.choice([1, 1, 2, 3, 5, 9]) for _ in range(rng.randint(1, 5))], stages
