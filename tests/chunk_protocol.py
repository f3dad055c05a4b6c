"""A CPU model of how the roles of cache_chunk_kernel wait for one another.

Load, softmax and product warps are generators that run in random order.  An
mbarrier is its phase counter and is waited for by parity alone, as in the
hardware; the tensor cores take the issued products one after another, at any
later time; a copy arrives when its warp waits for it, at the latest.  What
every step finds in shared memory and TMEM is checked against what it should
find there, and nothing may be written while something issued still reads it.

Faults: a load whose arrival is never reported, or waits that give up at random
(`spurious`).  A wait also gives up where nothing else can run, and may as soon
as another one has.  Mutants are protocols that are wrong in one place.
"""
import os
import random
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "clustered_multipole_approximation_b200", "csrc", "cache_chunk.cu")


def constants():
    """{(8-bit, D): stages}, copies ahead of a report (stages less) and scale slots, from the kernel's source."""
    src = open(SRC).read()
    ns = re.search(r"NS = CT == kCacheBf16 \? \(D == 128 \? (\d+) : (\d+)\) : \(D == 128 \? (\d+) : (\d+)\);", src)
    stages = dict(zip([(False, 128), (False, 64), (True, 128), (True, 64)], map(int, ns.groups())))
    lag = int(re.search(r"LAG = NS - (\d+);", src).group(1))
    scales = int(re.search(r"constexpr int kScales = (\d+);", src).group(1))
    return stages, lag, scales


class Wrong(Exception):
    pass


def check(cond, what):
    if not cond:
        raise Wrong(what)


class Bar:
    def __init__(self, count):
        self.count, self.n, self.phase = count, 0, 0

    def arrive(self):
        self.n += 1
        if self.n == self.count:
            self.n, self.phase = 0, self.phase + 1

    def passes(self, use):
        return (self.phase & 1) != (use & 1)


class Run:
    def __init__(self, nt, two, k8, stages, ahead, scales, seed, idle=(), lost=None, spurious=0.0, mutant=None):
        self.r = random.Random(seed)
        self.nt, self.two, self.k8, self.NS, self.ahead, self.scales = nt, two, k8, stages, ahead, scales
        self.idle, self.lost, self.spurious, self.mutant = idle, lost, spurious, mutant
        self.full = [Bar(4) for _ in range(stages)]
        self.empty = [Bar(1) for _ in range(stages)]
        self.S, self.O, self.done = [Bar(1), Bar(1)], [Bar(1), Bar(1)], Bar(1)
        self.P = [[Bar(4), Bar(4)], [Bar(4), Bar(4)]]
        self.stage = [[None] * 4 for _ in range(stages)]  # (load, arrived) of every load warp's share
        self.slot = [[None] * 4 for _ in range(scales)]   # tile of the scales
        self.s_tile = [None, None]                        # tile that S holds, by stream
        self.p_tile = [[[None] * 4, [None] * 4] for _ in range(2)]
        self.queue = []      # products and commits that were issued and have not run
        self.fail = False    # sfail
        self.lame = set()    # softmax warps behind a wait that gave up
        self.copies = set()  # on their way: (warp, load)
        self.finished = {}

    # the kernel's maps
    def n(self, w):
        return self.nt if self.two else (self.nt - w + 1) >> 1

    def tile(self, w, k):
        return k if self.two else 2 * k + w

    def k_item(self, t):
        return 0 if t == 0 else 2 * t - 1

    def v_item(self, t):
        return min(2 * t + 2, 2 * self.nt - 1)

    def is_k(self, i):
        return i == 0 or (i & 1 and i < 2 * self.nt - 1)

    def holds(self, st, item, what):
        check(all(x == (item, True) for x in self.stage[st]), what)

    # ---- load warps
    def begin_write(self, lw, item):
        st = item % self.NS
        check(not any(op[0] != "commit" and op[1] == st for op in self.queue), "a stage written under a product")
        self.stage[st][lw] = (item, False)

    def report(self, lw, item):
        st = item % self.NS
        check(self.stage[st][lw] == (item, True), "a load reported before it arrived")
        if item != self.lost:
            self.full[st].arrive()

    def landed(self, lw, upto):
        for lw2, item in sorted(self.copies):
            if lw2 == lw and item < upto:
                self.copies.discard((lw2, item))
                if self.stage[item % self.NS][lw][0] == item:
                    self.stage[item % self.NS][lw] = (item, True)

    def load8(self, lw):
        for item in range(2 * self.nt):
            if item >= self.NS:
                early = self.mutant == "a stage taken early"
                ok = yield self.empty[item % self.NS], item // self.NS - 1 - early
                if not ok and self.mutant != "load goes on":
                    return
            self.begin_write(lw, item)
            if self.is_k(item):
                self.slot[(item + 1) // 2 % self.scales][lw] = (item + 1) // 2
            yield None
            self.stage[item % self.NS][lw] = (item, True)
            self.report(lw, item)
            yield None

    def load16(self, lw):
        told = issued = 0
        lag = self.NS - self.ahead
        for item in range(2 * self.nt):
            if item >= self.NS and not self.empty[item % self.NS].passes(item // self.NS - 1):
                if self.mutant != "arrivals held back":
                    self.landed(lw, issued)
                    while told < issued:
                        self.report(lw, told)
                        told += 1
                ok = yield self.empty[item % self.NS], item // self.NS - 1
                if not ok:
                    return
            self.begin_write(lw, item)
            self.copies.add((lw, item))
            issued += 1
            yield None
            self.landed(lw, issued - lag)
            while told < issued - lag:
                self.report(lw, told)
                told += 1
        self.landed(lw, issued)
        while told < issued:
            self.report(lw, told)
            told += 1

    # ---- the product warp
    def issue_s(self, w, item, tile):
        self.queue.append(("S", item % self.NS, item, w, tile))
        self.queue.append(("commit", self.S[w]))
        if not self.two or w == (0 if self.mutant == "K freed early" else 1):
            self.queue.append(("commit", self.empty[item % self.NS]))

    def product(self):
        ok = True
        n = [self.n(0), self.n(1)]
        go = self.mutant == "products go on"
        for w in range(2):
            if n[w]:
                t = 0 if self.two else w
                item = self.k_item(t)
                ok = (ok and (yield self.full[item % self.NS], item // self.NS))
                if ok or go:
                    self.issue_s(w, item, t)
        for k in range(n[0]):
            for w in range(2):
                if k >= n[w]:
                    break
                T, more = self.tile(w, k), k + 1 < n[w]
                vi = self.v_item(T)
                ki = self.k_item(self.tile(w, k + 1)) if more else vi
                if not self.two or w == 0:
                    ok = ok and (yield self.full[vi % self.NS], vi // self.NS)
                    ok = ok and (yield self.full[ki % self.NS], ki // self.NS)
                for u in range(2):
                    ok = ok and (yield self.P[w][0 if self.mutant == "half of P" else u], k)
                    if not ok and not go:
                        continue
                    self.queue.append(("PV", vi % self.NS, vi, w, T, u))
                    if u and (not self.two or w == 1):
                        self.queue.append(("commit", self.empty[vi % self.NS]))
                    if u and not more:
                        self.queue.append(("commit", self.O[w]))
                if more and (ok or go):
                    self.issue_s(w, ki, self.tile(w, k + 1))
            if not ok and not go:
                break
        if self.mutant != "not drained" and (not ok or self.mutant != "drained by the product warp's waits alone"):
            self.queue.append(("commit", self.done))
            while not self.done.passes(0):  # the tensor cores always finish
                yield None

    def tensor_core(self):
        op = self.queue.pop(0)
        if op[0] == "commit":
            op[1].arrive()
            return
        self.holds(op[1], op[2], "a product over a stage that holds something else")
        w, tile = op[3], op[4]
        if op[0] == "S":
            self.s_tile[w] = tile
        else:
            half = self.p_tile[w][op[5]]
            check(all(x == tile for i, x in enumerate(half) if (w, i) not in self.idle + tuple(self.lame)),
                  "P of another tile")

    # ---- softmax warps
    def look(self, T):
        if self.k8 and self.r.random() < 0.5 or self.r.random() < 0.6:  # tiles inside every row's range
            return True
        vi = self.v_item(T)
        ok = yield self.full[vi % self.NS], vi // self.NS + 2 * (self.mutant == "a phase too far")
        if ok:
            self.holds(vi % self.NS, vi, "looked at a stage that holds something else")
            yield None
            self.holds(vi % self.NS, vi, "a stage changed under a look")
        return ok

    def softmax(self, w, i):
        ok, idle = True, (w, i) in self.idle
        for k in range(self.n(w)):
            if not ok:  # (warps with rows end the step in which a wait gave up: they vote once a step)
                break
            T = self.tile(w, k)
            ok = yield self.S[w], k
            if idle and not ok:
                break

            def sees(cond, what):  # once a wait gave up the warp's rows are NaN, whatever it saw
                check(cond or not ok, what)

            def scales():
                sees(not self.k8 or idle or all(x == T for x in self.slot[T % self.scales]), "scales of another tile")

            sees(self.s_tile[w] == T, "S of another tile")
            scales()
            if ok:
                ok = yield from self.look(T)
            if not ok:
                self.lame.add((w, i))
            if k and self.r.random() < 0.4 and not idle:  # the maximum moves: O is rescaled
                sees(not any(op[0] == "PV" and op[3] == w for op in self.queue), "O rescaled under a product")
            for u in range(2):
                yield None
                scales()
                sees(idle or self.s_tile[w] == T, "S overwritten before it was read")
                self.p_tile[w][u][i] = T
                if ok or self.mutant == "P without S":
                    self.P[w][u].arrive()
        if ok and self.n(w):
            ok = yield self.O[w], 0
        self.finished["soft", w, i] = ok

    def go(self):
        """"done", or "failed" where a wait gave up and everything was put away."""
        roles = {("load", i): (self.load8 if self.k8 else self.load16)(i) for i in range(4)} if self.nt else {}
        roles["product"] = self.product()
        for w in range(2):
            for i in range(4):
                roles["soft", w, i] = self.softmax(w, i)
        wait = dict.fromkeys(roles)
        rows = good = False
        while roles:
            free = [p for p in roles if wait[p] is None or wait[p][0].passes(wait[p][1])]
            if self.fail or self.r.random() < self.spurious:
                some = [p for p in roles if p not in free]
                if some and self.r.random() < 0.3:
                    free.append(self.r.choice(some))
            if self.queue and (not free or self.r.random() < 0.3):
                self.tensor_core()
                continue
            if not free:
                check(self.lost is not None or self.fail or self.spurious, "every role waits")
                free = list(roles)  # half a second later
            p = self.r.choice(free)
            try:
                if wait[p] is None:
                    wait[p] = next(roles[p])
                else:
                    bar, use = wait[p]
                    ok = bar.passes(use)
                    check(not ok or bar.phase > use, "a wait passed by an earlier phase")
                    if not ok:
                        self.fail = True
                    wait[p] = roles[p].send(ok)
            except StopIteration:
                del roles[p]
            if not rows and len(self.finished) == 8:
                rows = True
                good = all(self.finished.values())
                if good:  # the epilogue writes rows over the stages
                    check(not any(op[0] != "commit" for op in self.queue) and not self.copies,
                          "rows written under a product or a copy")
        # the last barrier: TMEM is freed and the CTA ends
        check(not any(op[0] != "commit" for op in self.queue), "TMEM freed under a product")
        check(not self.copies, "a copy on its way at the CTA's end")
        check(good or self.fail, "a failure without the flag")
        return "done" if good else "failed"
