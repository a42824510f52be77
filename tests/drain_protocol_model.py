"""Host-side models of the tcgen05 products and attention gradient: what their waits cover, and how they end --
nothing may be in flight when a CTA releases its memory.

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
        self.bars, self.roles, self.pending, self.producers = {}, {}, [], set()
        self.flags = {0: False}          # abort flags by CTA
        self.cta = {}                    # a role's CTA, 0 unless named

    @property
    def abort(self):
        return any(self.flags.values())

    def bar(self, name, count):
        self.bars[name] = Bar(count)

    def copy(self, issuer, fn):          # a TMA load: lands in any order
        self.pending.append(("tma " + issuer, fn))

    def commit(self, issuer, fn):        # an MMA issuer's commit: in order
        self.pending.append(("mma " + issuer, fn))

    def _value(self, role, want):
        kind = want[0]
        if kind == "until":
            return True if want[1]() else None
        if self.bars[want[1]].passed(want[2]):
            return True
        return False if kind == "wait" and self.flags[self.cta.get(role, 0)] else None

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
            blocked = [k for k in live if want[k][0] == "wait" and self._value(k, want[k]) is None]
            if blocked and (gone or not self.late) and self.rng.random() < self.timeout_p:
                self.flags[self.cta.get(self.rng.choice(blocked), 0)] = True
                continue
            choices = [("role", k) for k in live if self._value(k, want[k]) is not None]
            copies = [i for i, (who, _) in enumerate(self.pending) if who.startswith("tma ")]
            if not (self.late and choices):      # late: copies land when nothing else can move
                choices += [("land", i) for i in copies]
            firsts = {}
            for i, (who, _) in enumerate(self.pending):
                if who.startswith("mma "):
                    firsts.setdefault(who, i)
            choices += [("land", i) for i in firsts.values()]
            if not choices:
                stuck = "; ".join(f"{k}: {want[k][0]} {want[k][1:]}" for k in live)
                if not blocked:
                    raise Hazard("a wait on the way out waits for nothing: " + stuck)
                self.flags[self.cta.get(self.rng.choice(blocked), 0)] = True     # a bounded wait runs out
                continue
            kind, who = self.rng.choice(choices)
            if kind == "role":
                step(who, self._value(who, want[who]))
            else:
                self.pending.pop(who)[1]()
        raise Hazard("step limit")


def gemm(kblocks, stages, rng, timeout_p=0.0, late=False, drain="always", hold=False):
    """gemm_kernel<false, BN>: tiles of kblocks[n] k blocks through `stages` stages and two accumulators, with a
    producer, an MMA issuer and epilogue warps (two here). drain: "always" (the kernel), "flag" (only if the
    abort flag is up when the producer leaves) or "never". hold: the epilogue waits for an arrival nothing makes."""
    s = Sim(rng, timeout_p, late)
    n_ep = 2
    for i in range(stages):
        s.bar(f"FULL{i}", 1)
        s.bar(f"EMPTY{i}", 1)
    for i in range(2):
        s.bar(f"AFULL{i}", 2 if hold else 1)
        s.bar(f"AEMPTY{i}", n_ep)
    s.bar("DRAIN", 1)
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
            check(acc[ab] == n, "the epilogue reads another tile's accumulator")
            stored[ab] += 1
            B[f"AEMPTY{ab}"].arrive()

    s.roles = {"producer": producer(), "mma": mma(), **{f"epilogue {i}": epilogue() for i in range(n_ep)}}
    s.producers = {"producer"}
    return s.run()


def gemm_pair(kblocks, rng, stages=3, timeout_p=0.0, late=False, hold=False):
    """gemm_pair_kernel: two CTAs, each with a producer and epilogue warps (two here); CTA 0 issues. Both CTAs' loads
    count on CTA 0's full barriers, its commits arrive in both CTAs. A producer stays until its last stages have
    been used or, after a wait that ran out, until its copies have landed (the kernel: a time far above theirs)."""
    s = Sim(rng, timeout_p, late)
    s.flags = {0: False, 1: False}
    n_ep, B = 2, s.bars
    for i in range(stages):
        s.bar(f"FULL{i}", 3)                     # the announcement of the bytes, and each CTA's copies
        for r in range(2):
            s.bar(f"EMPTY{r}{i}", 1)
    for i in range(2):
        s.bar(f"AEMPTY{i}", 2 * n_ep)
        for r in range(2):
            s.bar(f"AFULL{r}{i}", 2 if hold else 1)
    s.bar("DRAIN", 1)
    held, used, acc, stored = [[None] * stages for _ in range(2)], [-1], [None, None], [0, 0]

    def producer(r):
        it, ok = 0, True
        for n in range(len(kblocks)):
            for _ in range(kblocks[n]):
                st = it % stages
                ok = ok and (yield "wait", f"EMPTY{r}{st}", ((it // stages) & 1) ^ 1)
                if not ok:
                    break
                check(used[0] >= it - stages, "a stage is filled before its products have read it")
                if r == 0:
                    B[f"FULL{st}"].arrive()

                def land(st=st, it=it):
                    held[r][st] = it
                    B[f"FULL{st}"].arrive()
                s.copy(f"p{r}", land)
                it += 1
        for j in range(max(0, it - stages), it):
            ok = ok and (yield "wait", f"EMPTY{r}{j % stages}", (j // stages) & 1)
        if not ok:
            yield "until", lambda: not any(who == f"tma p{r}" for who, _ in s.pending)

    def mma():
        it, ok = 0, True
        for n in range(len(kblocks)):
            ab = n & 1
            ok = ok and (yield "wait", f"AEMPTY{ab}", ((n >> 1) & 1) ^ 1)
            if not ok:
                break
            check(n < 2 or stored[ab] == 2 * n_ep * (n // 2), "an accumulator is overwritten before it is read")
            for _ in range(kblocks[n]):
                st = it % stages
                ok = yield "wait", f"FULL{st}", (it // stages) & 1
                if not ok:
                    break
                check(held[0][st] == it and held[1][st] == it, "a product reads a stage that holds something else")

                def done(st=st, it=it):
                    used[0] = it
                    B[f"EMPTY0{st}"].arrive()
                    B[f"EMPTY1{st}"].arrive()
                s.commit("m", done)
                it += 1
            if ok:
                def full(ab=ab, n=n):
                    acc[ab] = n
                    B[f"AFULL0{ab}"].arrive()
                    B[f"AFULL1{ab}"].arrive()
                s.commit("m", full)
        s.commit("m", B["DRAIN"].arrive)
        yield "drain", "DRAIN", 0

    def epilogue(r):
        for n in range(len(kblocks)):
            ab = n & 1
            if not (yield "wait", f"AFULL{r}{ab}", (n >> 1) & 1):
                return
            check(acc[ab] == n, "the epilogue reads another tile's accumulator")
            stored[ab] += 1
            B[f"AEMPTY{ab}"].arrive()

    s.roles = {"mma": mma(), **{f"producer {r}": producer(r) for r in range(2)},
               **{f"epilogue {r}.{i}": epilogue(r) for r in range(2) for i in range(n_ep)}}
    s.cta = {name: 1 for name in s.roles if name.startswith(("producer 1", "epilogue 1"))}
    s.producers = {"producer 0", "producer 1"}
    return s.run()


def random_gemm(rng):
    stages = rng.choice([2, 3, 6])
    return [rng.choice([1, 1, 2, 3, 5, 9]) for _ in range(rng.randint(1, 5))], stages


def bwd_slot(d, key, g, is_x):
    """Slot and use count of pair g's X or Y (attn_bwd.cu's slot_of)."""
    if d == 64:
        return 2 * (g % 4) + is_x, g // 4
    if key:
        n = 2 * g + (0 if is_x else 1)
        return n % 5, n // 5
    return (g % 3, g // 3) if is_x else (3 + g % 2, g // 2)


def bwd_last_use(d, key, g, is_x, gx, gy):
    """attn_bwd.cu's last_use."""
    if d == 64:
        return g + 4 >= (gx if is_x else gy)
    if key:
        return g + 2 >= gy if is_x else g + 3 >= gx
    return g + 3 >= gx if is_x else g + 2 >= gy


def bwd_pass(d, key, items, rng, timeout_p=0.0, late=False, drain="always", hold=False, first="free"):
    """One pass of attn_bwd_kernel over items given as their numbers of streamed pairs: the producer warp with its
    X and Y lanes, the issuers of S, dP, acc1 and (key pass) acc0, and the warps that turn S and dP into P and dS
    (two here). drain: "always" (the kernel), "flag" (only if the abort flag is up when the producer leaves,
    and for the last four loads of a lane whatever has used their slots since) or "never". first: what the issuers of
    S and dP wait for first, "free" (the kernel: their buffer's release) or "full" (their tile)."""
    s = Sim(rng, timeout_p, late)
    B, n_wg, n_iss, bufs = s.bars, 2, 4 if key else 3, 1 if d == 128 else 2
    for i in range(8):
        s.bar(f"FULL{i}", 1)
        s.bar(f"EMPTY{i}", 2 if d == 64 and key else 1)
    for i in range(2):
        for name, count in (("SFULL", 3 if hold else 2), ("SFREE", n_wg), ("IFULL", 1), ("IEMPTY", n_iss + n_wg), ("PREADY", n_wg),
                            ("PFREE", n_iss - 2)):
            s.bar(f"{name}{i}", count)
    for name, count in (("STATFULL", 1), ("STATEMPTY", 2), ("ACCFULL", n_iss - 2), ("ACCFREE", n_wg), ("COLS", n_wg),
                        ("DRAIN", n_iss)):
        s.bar(name, count)
    info, pairs = [None, None], [None] * 4
    held, stat = [None] * 8, [None]             # what the slots and the stationary tiles hold
    g = {True: 0, False: 0}                      # pairs issued by the X and the Y lane
    lanes = {"it": -1, True: None, False: None}  # the item at work; whether a lane is through (its ok)
    sbuf, pbuf = [[None, None], [None, None]], [None, None]
    done = {"S": -1, "dP": -1, "acc1": -1, "acc0": -1}       # last pair of each product that has completed
    read = {"acc": -1, "s": [0, 0]}

    def producer():
        ok, stat_it = True, -1
        for it in range(len(items) + 1):
            slot = it & 1
            if not (ok := (yield "wait", f"IEMPTY{slot}", ((it >> 1) & 1) ^ 1)):
                break
            info[slot] = (it, items[it]) if it < len(items) else (it, None)
            B[f"IFULL{slot}"].arrive()
            if it == len(items):
                break
            ok = yield "wait", "STATEMPTY", (it & 1) ^ 1
            if ok:
                if items[it] or drain != "flag":         # the flag form counted only the items with loads
                    stat_it = it
                if items[it]:
                    def land(it=it):
                        stat[0] = it
                        B["STATFULL"].arrive()
                    s.copy("stat", land)
                else:
                    B["STATFULL"].arrive()
            lanes[True] = lanes[False] = None
            lanes["ok"], lanes["it"] = ok, it
            yield "until", lambda: lanes[True] is not None and lanes[False] is not None
            ok = lanes[True] and lanes[False]
            if not ok:
                break
        lanes["it"] = len(items)                          # the lanes leave
        if drain == "never" or (drain == "flag" and not s.abort):
            return
        if stat_it >= 0:
            yield "drain", "STATFULL", stat_it & 1
        for x in (True, False):
            for j in range(max(0, g[x] - 4), g[x]):
                slot, use = bwd_slot(d, key, j, x)
                if drain == "flag" or bwd_last_use(d, key, j, x, g[True], g[False]):
                    yield "drain", f"FULL{slot}", use & 1

    def lane(x):
        for it in range(len(items)):
            yield "until", lambda it=it: lanes["it"] >= it
            if lanes["it"] == len(items):
                return
            ok = lanes["ok"]
            for j in range(items[it]):
                if not ok:
                    break
                slot, use = bwd_slot(d, key, g[x], x)
                ok = yield "wait", f"EMPTY{slot}", (use & 1) ^ 1
                if not ok:
                    break
                if held[slot] is not None:
                    gg, xx = held[slot]
                    users = [p for p in ("S" if xx else "dP", "acc1" if xx else "acc0")
                             if p != "acc0" or key]
                    if d == 64:
                        users = ["acc1", "acc0"] if key else ["acc1"]
                    check(all(done[p] >= gg for p in users), f"slot {slot} is filled before pair {gg} is used")
                if x:
                    pairs[g[x] & 3] = g[x]

                def land(slot=slot, gg=g[x]):
                    held[slot] = (gg, x)
                    B[f"FULL{slot}"].arrive()
                s.copy("x" if x else "y", land)
                g[x] += 1
            lanes[x] = ok

    def issuer_s(name):
        x, gi = name == "S", 0
        for it in range(len(items) + 1):
            slot = it & 1
            if not (yield "wait", f"IFULL{slot}", (it >> 1) & 1):
                break
            got, n = info[slot]
            check(got == it, f"{name} took item {got} for {it}")
            B[f"IEMPTY{slot}"].arrive()
            if n is None:
                break
            if not (yield "wait", "STATFULL", it & 1):
                break
            ok = True
            for _ in range(n):
                b, (sl, use) = gi & 1, bwd_slot(d, key, gi, x)
                waits = [("wait", f"SFREE{b}", ((gi >> 1) & 1) ^ 1), ("wait", f"FULL{sl}", use & 1)]
                for w in waits if first == "free" else waits[::-1]:
                    ok = ok and (yield w)
                if not ok:
                    break
                check(stat[0] == it and held[sl] == (gi, x), f"{name}({gi}) reads another tile")
                check(gi < 2 or read["s"][b] == n_wg * (gi // 2), f"{name}({gi}) overwrites a buffer before it is read")

                def land(gi=gi, b=b, sl=sl):
                    sbuf[b][x], done[name] = gi, gi
                    B[f"SFULL{b}"].arrive()
                s.commit(name, land)
                if not key and d == 128 and not x:
                    s.commit(name, B[f"EMPTY{sl}"].arrive)
                gi += 1
            if not ok:
                break
            s.commit(name, B["STATEMPTY"].arrive)
        s.commit(name, B["DRAIN"].arrive)
        yield "drain", "DRAIN", 0

    def issuer_acc(name):
        x, gi = name == "acc1" and d == 128, 0
        for it in range(len(items) + 1):
            slot = it & 1
            if not (yield "wait", f"IFULL{slot}", (it >> 1) & 1):
                break
            got, n = info[slot]
            check(got == it, f"{name} took item {got} for {it}")
            B[f"IEMPTY{slot}"].arrive()
            if n is None:
                break
            if not (yield "wait", "ACCFREE", (it & 1) ^ 1):
                break
            check(read["acc"] >= it - 1, f"{name} overwrites gradients that are not read")
            ok = True
            for _ in range(n):
                sl, use = bwd_slot(d, key, gi, x)
                pb = gi % bufs
                ok = yield "wait", f"FULL{sl}", use & 1
                ok = ok and (yield "wait", f"PREADY{pb}", (gi // bufs) & 1)
                if not ok:
                    break
                check(pbuf[pb] == gi and held[sl] == (gi, x), f"{name}({gi}) reads another pair")
                check(d == 128 or held[sl + 1] == (gi, True), f"{name}({gi}) reads another X")

                def land(gi=gi, pb=pb, sl=sl):
                    done[name] = gi
                    B[f"PFREE{pb}"].arrive()
                    B[f"EMPTY{sl}"].arrive()
                    if d == 64:
                        B[f"EMPTY{sl + 1}"].arrive()
                s.commit(name, land)
                gi += 1
            if not ok:
                break
            s.commit(name, B["ACCFULL"].arrive)
        s.commit(name, B["DRAIN"].arrive)
        yield "drain", "DRAIN", 0

    finished, ready = {}, {}

    def warp(w):
        gi = 0
        for it in range(len(items) + 1):
            slot = it & 1
            if not (yield "wait", f"IFULL{slot}", (it >> 1) & 1):
                return
            got, n = info[slot]
            check(got == it, f"a warp took item {got} for {it}")
            B[f"IEMPTY{slot}"].arrive()
            if n is None:
                return
            if not key:
                B["COLS"].arrive()
                if not (yield "wait", "COLS", it & 1):
                    return
            for _ in range(n):
                b, (sl, use), pb = gi & 1, bwd_slot(d, key, gi, True), gi % bufs
                if not (yield "wait", f"FULL{sl}", use & 1):
                    return
                check(pairs[gi & 3] == gi, "a warp reads another pair's tiles")
                if not (yield "wait", f"SFULL{b}", (gi >> 1) & 1):
                    return
                check(sbuf[b] == [gi, gi], f"a warp reads another pair's S or dP for {gi}")
                read["s"][b] += 1
                B[f"SFREE{b}"].arrive()
                if not (yield "wait", f"PFREE{pb}", ((gi // bufs) & 1) ^ 1):
                    return
                check(min(done[a] for a in (("acc1", "acc0") if key else ("acc1",))) >= gi - bufs,
                      "P is overwritten before its products have read it")
                ready[gi] = ready.get(gi, 0) + 1
                if ready[gi] == n_wg:
                    pbuf[pb] = gi
                B[f"PREADY{pb}"].arrive()
                gi += 1
            if not (yield "wait", "ACCFULL", it & 1):
                return
            check(n == 0 or min(done[a] for a in (("acc1", "acc0") if key else ("acc1",))) >= gi - 1,
                  "gradients are read before they are complete")
            finished[it] = finished.get(it, 0) + 1
            if finished[it] == n_wg:
                read["acc"] = it
            B["ACCFREE"].arrive()

    s.roles = {"producer": producer(), "lane x": lane(True), "lane y": lane(False), "S": issuer_s("S"), "dP": issuer_s("dP"),
               "acc1": issuer_acc("acc1"), **({"acc0": issuer_acc("acc0")} if key else {}),
               **{f"warp {w}": warp(w) for w in range(n_wg)}}
    s.producers = {"producer", "lane x", "lane y"}
    return s.run()


def random_items(rng):
    return [rng.choice([0, 1, 1, 2, 3, 5, 8]) for _ in range(rng.randint(1, 5))]
