"""The warp roles and barriers of csrc/paged_attend_tc.cu as coroutines, run in random orders.

One CTA: the walker, the K and V loaders, the MMA issuer, 16 softmax warps, the asynchronous
copies and the tensor core.  A wait that nothing will satisfy any more ends a run as `Stuck`;
every buffer carries the piece and step that it holds, so an early overwrite ends it as an
AssertionError.  Barriers are waited for by parity, as the hardware does: a waiter that two
phases have passed by waits for a third.
"""

import random

NSLOT, NSB = 8, 3
QUADS, PARTS = 4, 4  # 32-row groups; softmax warps of each (two of the even steps' group, two of the odd one's)


class Stuck(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        assert self.pending >= 0
        self.turn()

    def land(self):
        self.tx -= 1
        self.turn()

    def turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):
        return self.phase & 1 != parity


class Cta:
    """pieces: a list of (steps, fixed, exchanged): its steps; those of them whose V rows get zeros;
    the quads whose warps exchange the largest scores of the first step (all four without a cap).

    tops_by: how the barrier of that exchange is used: "two", two a quad, by the number of the
    exchange; "one", one a quad, which is too few.  drains: "issued", the V loader's exit waits for
    copies of zeroed rows that it issued; "always", whether or not there are any.  gives_up: after
    so many waits one of them runs into its limit."""

    def __init__(self, pieces, HD, rng, tops_by="two", drains="issued", gives_up=None):
        self.pieces, self.rng, self.tops_by, self.drains, self.gives_up = pieces, rng, tops_by, drains, gives_up
        stages = 4 if HD == 64 else 2
        bars = lambda n, count: [Bar(count) for _ in range(n)]  # noqa: E731
        self.qfull, self.qempty = bars(2, 1), bars(2, 1)
        self.kfull, self.kempty, self.vfull, self.vempty = (bars(stages, 1) for _ in range(4))
        self.sfull, self.pfull = bars(NSB, 1), bars(NSB, QUADS * PARTS // 2)
        self.ofull, self.oempty, self.vfix, self.final = Bar(1), Bar(QUADS * PARTS), Bar(1), Bar(1)
        self.ifull, self.iempty = bars(NSLOT, 1), bars(NSLOT, 3 + QUADS * PARTS)
        self.sums_bar = bars(QUADS, PARTS)
        self.tops_bar = bars(2 * QUADS, PARTS // 2)
        self.items, self.q, self.k, self.v = [None] * NSLOT, [None] * 2, [None] * stages, [None] * stages
        self.s, self.p = [None] * NSB, [set() for _ in range(NSB)]  # what a score buffer holds; P's parts
        self.o, self.o_read = None, QUADS * PARTS
        self.sums = [[[None] * QUADS for _ in range(PARTS)] for _ in range(2)]
        self.bad = [[[None] * QUADS for _ in range(PARTS)] for _ in range(2)]
        self.tops = [[[None] * QUADS for _ in range(2)] for _ in range(2)]
        self.drained = [[0] * QUADS for _ in range(2)]
        self.results = [[0] * QUADS for _ in pieces]
        self.copies, self.mmas, self.abort, self.waits = [], [], False, 0

    # ------------------------------------------------------------ the roles
    # A role yields (barrier, parity) to wait, with False for a wait that gave up; (barrier,
    # parity, "drain") for one that abort does not end; None to let others go on.
    def piece(self, k):
        if not (yield self.ifull[k % NSLOT], k // NSLOT & 1):
            return None
        tag, x = self.items[k % NSLOT]
        assert tag == k
        return x

    def walker(self):
        loaded = 0
        for k, x in enumerate(self.pieces + [None]):
            if k >= NSLOT and not (yield self.iempty[k % NSLOT], k // NSLOT - 1 & 1):
                break
            self.items[k % NSLOT] = k, x
            self.ifull[k % NSLOT].arrive()
            yield None
            if x is None:
                break
            if k >= 2 and not (yield self.qempty[k & 1], (k >> 1) - 1 & 1):
                break
            self.qfull[k & 1].arrive(tx=1)
            self.copies.append((self.qfull[k & 1], self.q, k & 1, k))
            loaded = k + 1
            yield None
        for x in range(max(0, loaded - 2), loaded):
            yield self.qfull[x & 1], x >> 1 & 1, "drain"

    def loader(self, values):
        tiles, full, empty = (self.v, self.vfull, self.vempty) if values else (self.k, self.kfull, self.kempty)
        stages, j, fixes, ok, landing, k = len(tiles), 0, 0, True, False, 0
        while ok:
            x = yield from self.piece(k)
            if x is None:
                break
            steps, fixed, _ = x
            self.iempty[k % NSLOT].arrive()
            for i in range(steps):
                s, u = j % stages, j // stages
                if u > 0 and not (yield empty[s], u - 1 & 1):
                    ok = False
                    break
                fix = values and i in fixed
                bar = self.vfix if fix else full[s]
                bar.arrive(tx=1)
                self.copies.append((bar, tiles, s, (k, i)))
                yield None
                if fix:
                    if not (yield self.vfix, fixes & 1):
                        ok, landing = False, True
                        break
                    fixes += 1
                    full[s].arrive()
                j += 1
            k += 1
        if values and not ok and (landing or self.drains == "always"):
            yield self.vfix, fixes & 1, "drain"
        for x in range(max(0, j - stages), j):
            yield full[x % stages], x // stages & 1, "drain"

    def issuer(self):
        at = dict(k=0, left=0, g=0, stage=0, phase=0, i=0)

        def scores():
            if at["left"] == 0:
                if not (yield self.ifull[at["k"] % NSLOT], at["k"] // NSLOT & 1):
                    return -1
                tag, x = self.items[at["k"] % NSLOT]
                assert tag == at["k"]
                if x is None:
                    return 0
                at["left"], at["i"] = x[0], 0
                if not (yield self.qfull[at["k"] & 1], at["k"] >> 1 & 1):
                    return -1
            if not (yield self.kfull[at["stage"]], at["phase"]):
                return -1
            self.mmas.append(("S", at["g"], at["k"] & 1, at["stage"], (at["k"], at["i"])))
            self.mmas += [("commit", self.sfull[at["g"]]), ("commit", self.kempty[at["stage"]])]
            at["left"] -= 1
            at["i"] += 1
            if at["left"] == 0:
                self.mmas.append(("commit", self.qempty[at["k"] & 1]))
                at["k"] += 1
            at["g"] = (at["g"] + 1) % NSB
            at["stage"] += 1
            if at["stage"] == len(self.k):
                at["stage"], at["phase"] = 0, at["phase"] ^ 1
            yield None
            return 1

        ahead, k = 1, 0
        for _ in range(NSB):
            if ahead > 0:
                ahead = yield from scores()
        g = gp = vs = vp = 0
        while ahead >= 0:
            x = yield from self.piece(k)
            if x is None:
                break
            ok = True
            for i in range(x[0]):
                ok = (yield self.pfull[g], gp) and (yield self.vfull[vs], vp)
                if ok and i == 0 and k > 0:
                    ok = yield self.oempty, k - 1 & 1
                if not ok:
                    break
                self.mmas += [("PV", g, vs, (k, i)), ("commit", self.vempty[vs])]
                if i + 1 == x[0]:
                    self.mmas.append(("commit", self.ofull))
                yield None
                g, gp = (g + 1, gp) if g + 1 < NSB else (0, gp ^ 1)
                vs, vp = (vs + 1, vp) if vs + 1 < len(self.v) else (0, vp ^ 1)
                if ahead > 0:
                    ahead = yield from scores()
                ok = ahead >= 0
                if not ok:
                    break
            self.iempty[k % NSLOT].arrive()
            k += 1
            if not ok:
                break
        self.mmas.append(("commit", self.final))
        yield self.final, 0, "drain"

    def softmax(self, cq, quad):
        group, half = cq >> 1, cq & 1
        at = dict(sb=group, sp=0, exchanges=0)

        def drain(k):
            xx = k & 1
            if not (yield self.ofull, k & 1):
                return False
            assert self.o == (k, self.pieces[k][0] - 1)
            yield None
            self.o_read += 1
            self.oempty.arrive()
            yield None
            self.bad[xx][cq][quad] = k
            self.drained[xx][quad] += 1
            last = self.drained[xx][quad] == PARTS
            if last:
                self.drained[xx][quad] = 0
            yield None
            if not (yield self.sums_bar[quad], k & 1):
                return False
            yield None
            assert all(self.sums[xx][e][quad] == k for e in range(PARTS))
            if last:
                assert all(self.bad[xx][e][quad] == k for e in range(PARTS))
                self.results[k][quad] += 1
            yield None  # stores
            self.iempty[k % NSLOT].arrive()
            return True

        def tops_of(k):
            x = at["exchanges"]
            if self.tops_by == "one":
                return self.tops_bar[quad], x & 1, x & 1
            return self.tops_bar[2 * quad + (x & 1)], x >> 1 & 1, x & 1

        def reference(k):
            bar, parity, buffer = tops_of(k)
            if not (yield bar, parity):
                return False
            yield None
            assert all(self.tops[buffer][h][quad] == k for h in range(2))
            at["exchanges"] += 1
            return True

        def step(k, i, exchanged):
            sb = at["sb"]
            if not (yield self.sfull[sb], at["sp"]):
                return False
            assert self.s[sb] == (k, i)
            if i == 0 and quad in exchanged:
                bar, _, buffer = tops_of(k)
                self.tops[buffer][half][quad] = k
                yield None
                bar.arrive()
                if not (yield from reference(k)):
                    return False
            yield None
            assert self.s[sb] == (k, i)
            self.p[sb].add((half, quad))
            self.pfull[sb].arrive()
            at["sb"] = sb + 2
            if at["sb"] >= NSB:
                at["sb"] -= NSB
                at["sp"] ^= 1
            return True

        g = k = 0
        while True:
            x = yield from self.piece(k)
            if x is None and (k == 0 or self.abort):
                break
            n, _, exchanged = x or (0, (), ())
            ok, i = True, 0 if x is not None and g & 1 == group else -1
            while ok and i < max(n, 1):
                if 0 <= i < n:
                    ok = yield from step(k, i, exchanged)
                if i <= 0:
                    if ok and k > 0:
                        ok = yield from drain(k - 1)
                    if x is None:
                        break
                    if quad in exchanged and i < 0:
                        ok = ok and (yield from reference(k))
                i += 2
            if not ok or x is None:
                break
            g += n
            self.sums[k & 1][cq][quad] = k
            self.sums_bar[quad].arrive()
            yield None
            k += 1

    # ------------------------------------------------------------ copies, products, the order
    def land(self):
        bar, tiles, at, what = self.copies.pop(self.rng.randrange(len(self.copies)))
        tiles[at] = what
        bar.land()

    def product(self):
        op = self.mmas.pop(0)
        if op[0] == "commit":
            op[1].arrive()
        elif op[0] == "S":
            _, g, q, stage, (k, i) = op
            assert self.q[q] == k and self.k[stage] == (k, i) and self.s[g] is None
            self.s[g] = k, i
        else:
            _, g, stage, (k, i) = op
            assert self.s[g] == (k, i) and len(self.p[g]) == 2 * QUADS and self.v[stage] == (k, i)
            if i == 0:
                assert self.o_read == QUADS * PARTS
                self.o_read = 0
            else:
                assert self.o == (k, i - 1)
            self.o, self.s[g], self.p[g] = (k, i), None, set()

    def run(self):
        """To the end, in a random order: each role has a pace, and may stall for long."""
        rng = self.rng
        roles = [self.walker(), self.loader(False), self.loader(True), self.issuer()]
        roles += [self.softmax(cq, quad) for cq in range(PARTS) for quad in range(QUADS)]
        state = [next(r) for r in roles]  # what each waits for
        pace = [rng.choice([1, 1, 3, 20]) for _ in roles] + [rng.choice([1, 3, 20]) for _ in range(2)]
        slow = [0] * len(roles)
        while True:
            live = [r for r, w in enumerate(state) if w != "ended"]
            if not live and not self.mmas and not self.copies:
                return
            can = [r for r in live if state[r] is None or state[r][0].done(state[r][1]) or (self.abort and len(state[r]) == 2)]
            choice = [r for r in can if slow[r] == 0]
            choice += [len(roles)] * bool(self.copies) + [len(roles) + 1] * bool(self.mmas)
            slow = [max(0, n - 1) for n in slow]
            if not choice:
                if not can:
                    raise Stuck(live)
                continue
            r = rng.choices(choice, [pace[c] for c in choice])[0]
            if r == len(roles):
                self.land()
                continue
            if r == len(roles) + 1:
                self.product()
                continue
            if rng.random() < 0.01:
                slow[r] = rng.choice([20, 200])
            answer = None
            if state[r] is not None:
                answer = state[r][0].done(state[r][1])
                if len(state[r]) == 2:
                    self.waits += 1
                    if self.waits == self.gives_up:
                        answer, self.abort = False, True
            try:
                state[r] = roles[r].send(answer)
            except StopIteration:
                state[r] = "ended"


def random_pieces(rng, lengths, exchanged, count=12):
    """Pieces of these lengths; the first and last steps' V rows may get zeros."""
    out = []
    for _ in range(count):
        n = rng.choice(lengths)
        quads = range(QUADS) if exchanged == "all" else () if exchanged == "none" else \
            [q for q in range(QUADS) if rng.random() < 0.5]
        out.append((n, {i for i in (0, n - 1) if rng.random() < 0.5}, tuple(quads)))
    return out
