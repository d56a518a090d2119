"""The prompt kernel's barrier protocol, modelled on the CPU.

The loading thread, the two issuing warps, the warp that hands out units and looks over V tiles, and the softmax of the
two tiles run as processes in random interleavings over mbarriers, which a wait sees by the parity of a phase alone, as
the hardware's do.  Copies land in any order; MMAs and the commits behind them complete in the order of issue.  A unit
is (n, two): n steps of 128 keys, from the diagonal down, for one or two row tiles; step i's key tile is K(i), its value
tile V(i), and tile 0 of a unit of two starts with step 1.  The model checks that
  - a wait that returns has seen the phase it is for (parity alone does not tell a phase from the one two before);
  - every product reads the Q, K and V tile that it is meant for, whole and not yet overwritten;
  - the values of a unit's first two steps are looked over before a product reads them, and nothing else is;
  - all units end.
"""
import random

import pytest

STAGES = 4


class Bar:
    """An mbarrier: arrivals (expect-tx among them) and copies on their way, by phase."""

    def __init__(self, count):
        self.count, self.pend, self.tx, self.phase = count, count, 0, 0

    def arrive(self):
        assert self.pend > 0, "an arrival too many"
        self.pend -= 1
        self._check()

    def expect(self):
        self.tx += 1
        self.arrive()

    def land(self):
        self.tx -= 1
        self._check()

    def _check(self):
        if self.pend == 0 and self.tx == 0:
            self.phase += 1
            self.pend = self.count


def at_k(i):
    return 0 if i == 0 else 2 * i - 1


def at_v(i, n):
    return 2 * n - 1 if i == n - 1 else 2 * i + 2


class Block:
    """One block's roles.  own: the value tiles of a unit's first two steps land on barriers of their own, and who looks
    them over then completes their ring stages; otherwise they land on the ring's barriers, for which that warp waits as
    well.  part: tile 1's issuer takes part in units of one tile (sees and releases what they load); otherwise it passes
    over them and tile 0's issuer releases for both."""

    def __init__(self, units, own=True, part=True):
        self.units, self.own, self.part = units, own, part
        self.q_full, self.q_empty = Bar(1), Bar(2)
        self.full = [Bar(1) for _ in range(STAGES)]
        self.empty = [Bar(2) for _ in range(STAGES)]
        pair = lambda count: [Bar(count), Bar(count)]  # noqa: E731
        self.s_full, self.p_full, self.o_done, self.o_free, self.turn = pair(1), pair(1), pair(1), pair(1), pair(1)
        self.v_raw, self.v_ok = pair(1), [pair(1), pair(1)]
        self.unit_full, self.unit_empty = pair(1), pair(1 + 2 + 2)
        self.ring, self.q = [None] * STAGES, [None, None]
        self.looked = set()
        self.copies, self.pipe = [], []

    def unit(self, u):
        return self.units[u] if u < len(self.units) else (0, False)

    # -- roles: generators that yield (barrier, phase) to wait for
    def loader(self):
        c = 0
        for u in range(len(self.units) + 1):
            yield self.unit_full[u & 1], u >> 1
            n, two = self.unit(u)
            self.unit_empty[u & 1].arrive()
            if n == 0:
                return
            if u:
                yield self.q_empty, u - 1
            tiles = 1 + two
            for x in range(tiles):
                self.q[x] = None
            self.copy(self.q_full, [(self.q, x, ("q", u, x)) for x in range(tiles)])
            for pos in range(2 * n):
                is_v = pos == 2 * n - 1 or (pos > 0 and pos % 2 == 0)
                i = n - 1 if pos == 2 * n - 1 else pos // 2 - 1 if is_v else (pos + 1) // 2
                assert pos == (at_v(i, n) if is_v else at_k(i))
                st = c % STAGES
                if c >= STAGES:
                    yield self.empty[st], c // STAGES - 1
                self.ring[st] = None
                bar = self.v_raw[i] if self.own and is_v and i < 2 else self.full[st]
                self.copy(bar, [(self.ring, st, ("v" if is_v else "k", u, i))])
                c += 1

    def copy(self, bar, parts):
        bar.expect()
        bar.tx += len(parts) - 1
        self.copies += [(bar, *p) for p in parts]

    def issuer(self, x):
        base = steps = turns = mine = 0
        for u in range(len(self.units) + 1):
            yield self.unit_full[u & 1], u >> 1
            n, two = self.unit(u)
            self.unit_empty[u & 1].arrive()
            if n == 0:
                return
            if x == 1 and not two:
                if self.part:
                    yield self.q_full, u
                    self.q_empty.arrive()
                    for at in range(base, base + 2 * n):
                        yield self.full[at % STAGES], at // STAGES
                        self.empty[at % STAGES].arrive()
                base += 2 * n
                continue
            first_step = 1 if x == 0 and two else 0
            times = 2 if x == 0 and not two and not self.part else 1
            yield self.q_full, u
            for i in range(first_step - 1, n):
                more, first = i + 1 < n, i < first_step
                k, v = base + at_k(i + 1), base + at_v(max(i, 0), n)
                if more:
                    yield self.full[k % STAGES], k // STAGES
                if not first:
                    yield self.full[v % STAGES], v // STAGES
                    if i < 2 and not self.own:
                        yield self.v_ok[u & 1][i], u >> 1
                    if i == first_step and mine:
                        yield self.o_free[x], mine - 1
                    if two and (x == 0 or i > 0):
                        yield self.turn[x], turns
                        turns += 1
                    yield self.p_full[x], steps
                    steps += 1
                    self.pipe.append(("pv", x, v % STAGES, u, i))
                if more:
                    self.pipe.append(("qk", x, k % STAGES, u, i + 1))
                    if two and not first:
                        self.turn[x ^ 1].arrive()
                    self.pipe.append(("commit", self.s_full[x], 1))
                    if i + 2 == n:
                        self.pipe.append(("commit", self.q_empty, times))
                    self.pipe.append(("commit", self.empty[k % STAGES], times))
                else:
                    if x == 0 and two:
                        self.turn[1].arrive()
                    self.pipe.append(("commit", self.o_done[x], 1))
                if not first:
                    self.pipe.append(("commit", self.empty[v % STAGES], times))
                elif first_step == 1:
                    for at in (base, base + at_v(0, n)):
                        yield self.full[at % STAGES], at // STAGES
                        self.empty[at % STAGES].arrive()
            base += 2 * n
            mine += 1

    def looker(self):
        base = 0
        seen = [0, 0]                             # phases of v_raw
        for u in range(len(self.units) + 1):
            if u >= 2:
                yield self.unit_empty[u & 1], (u >> 1) - 1
            self.unit_full[u & 1].arrive()
            n, _ = self.unit(u)
            if n == 0:
                return
            for i in range(2):
                if i < n:
                    at = base + at_v(i, n)
                    if self.own:
                        yield self.v_raw[i], seen[i]
                        seen[i] += 1
                    else:
                        yield self.full[at % STAGES], at // STAGES
                    for _ in range(3):                # looking takes a while
                        self.sees(self.ring[at % STAGES], ("v", u, i))
                        yield None
                    self.looked.add((u, i))
                    if self.own:
                        self.full[at % STAGES].arrive()
                self.v_ok[u & 1][i].arrive()
            base += 2 * n

    def softmax(self, x):
        done = mine = 0
        for u in range(len(self.units) + 1):
            yield self.unit_full[u & 1], u >> 1
            n, two = self.unit(u)
            steps = 0 if n == 0 or (x == 1 and not two) else n - 1 if x == 0 and two else n
            for _ in range(steps):
                yield self.s_full[x], done
                done += 1
                self.p_full[x].arrive()
            if steps:
                yield self.o_done[x], mine
                mine += 1
                for i in range(2):
                    yield self.v_ok[u & 1][i], u >> 1
                self.o_free[x].arrive()
            self.unit_empty[u & 1].arrive()
            if n == 0:
                return

    @staticmethod
    def sees(found, meant):
        assert found == meant, f"finds {found} in the place of {meant}"

    def run(self, seed):
        rnd = random.Random(seed)
        roles = [self.loader(), self.issuer(0), self.issuer(1), self.looker(), self.softmax(0), self.softmax(1)]
        wait = [next(r) for r in roles]
        speed = [rnd.choice((1, 1, 4, 20)) for _ in range(8)]   # some interleavings are lopsided
        while True:
            acts = [k for k, w in enumerate(wait) if w is None or (w != "end" and (w[0].phase & 1) != (w[1] & 1))]
            acts += [6] * bool(self.copies) + [7] * bool(self.pipe)
            if not acts:
                assert all(w == "end" for w in wait), "deadlock"
                return
            a = rnd.choices(acts, [speed[k] for k in acts])[0]
            if a == 6:
                bar, place, at, what = self.copies.pop(rnd.randrange(min(len(self.copies), rnd.choice((1, 2, 8)))))
                place[at] = what
                bar.land()
            elif a == 7:
                op = self.pipe.pop(0)
                if op[0] == "commit":
                    for _ in range(op[2]):
                        op[1].arrive()
                else:
                    kind, x, st, u, i = op
                    self.sees(self.ring[st], (kind[1], u, i))
                    if kind == "qk":
                        self.sees(self.q[x], ("q", u, x))
                    else:
                        assert i >= 2 or (u, i) in self.looked, "values that were not looked over"
            else:
                if wait[a] is not None:
                    bar, phase = wait[a]
                    assert bar.phase > phase, f"role {a} takes phase {bar.phase - 2} for phase {phase}"
                wait[a] = next(roles[a], "end")


def units(seed):
    """The units of a block over packed prompts: 256 rows of one, or the up to 128 that are left of it, each with the
    keys up to them."""
    rnd = random.Random(seed)
    out = []
    for _ in range(rnd.randrange(2, 12)):
        two = rnd.random() < 0.5
        out.append((2 * rnd.choice((0, 0, 0, 1, 2, 5)) + 1 + two, two))
    return out


def test_every_wait_sees_its_own_phase():
    for seed in range(3000):
        Block(units(seed)).run(seed)


def test_looking_over_by_the_rings_barriers_breaks_it():
    """The warp that looks over V tiles runs up to a unit ahead of the ring: by parity it takes an earlier tile's phase
    for its own."""
    with pytest.raises(AssertionError, match="role 3 takes phase|finds"):
        for seed in range(1500):
            Block(units(seed), own=False).run(seed)


def test_an_issuer_that_passes_over_units_breaks_it():
    """It takes the Q of the unit that it passed over for the next one's, or a ring stage that is two phases behind."""
    with pytest.raises(AssertionError, match="role 2 takes phase"):
        for seed in range(3000):
            Block(units(seed), part=False).run(seed)
