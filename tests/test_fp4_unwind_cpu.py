"""How a CTA of the 4-bit grouped product (gemm_fp4.cu) ends when a wait gives up, modelled on the CPU.

The model holds barriers as the hardware does (arrivals still to come and a count of bytes), copies and
signals in flight that land at any time, and one thread's commits, which land in order.  One wait of one
role gives up on purpose; the others of its CTA end at their next wait that is not ready, and whatever is
then left waiting gives up in its turn, as the kernel's bounded waits do.  A CTA, and a pair as a whole,
may end only when nothing in flight reads or writes its shared memory any more."""

import random

import pytest

from test_fp4_pipeline_cpu import depths, tiles

BYTES = 100  # of one CTA's copies in a stage; signals carry SIGNAL
SIGNAL = 16


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.done = count, count, 0, 0

    def arrive(self, expect=0):
        self.pending -= 1
        self.change(expect)

    def change(self, tx):
        self.tx += tx
        assert self.pending >= 0
        if self.pending == 0 and self.tx == 0:
            self.pending, self.done = self.count, self.done + 1

    def ready(self, parity):
        return (self.done & 1) != parity


class Cluster:
    """One CTA or a pair, its roles under a random schedule."""

    def __init__(self, stages_of_tiles, pair, seed, give_up, rule):
        self.rng = random.Random(seed)
        self.n_codes, self.n_scales, self.turners = depths(pair)
        self.pair, self.rule, self.ctas = pair, rule, range(2 if pair else 1)
        self.tiles, self.total = stages_of_tiles, sum(stages_of_tiles)
        n = len(self.ctas)

        def ring(depth, count):
            return [[Barrier(count) for _ in range(depth)] for _ in self.ctas]

        self.full, self.turned = ring(self.n_codes, 1), ring(self.n_scales, 1)  # the leader's are used
        self.empty, self.sempty, self.sfull = ring(self.n_codes, 1), ring(self.n_scales, 1), ring(self.n_scales, 1)
        self.accf, self.acce, self.finished = ring(2, 1), ring(2, 2 * n), [Barrier(1)]
        self.abort, self.unwind = [False] * n, [False] * n
        self.issued, self.loaded = [0] * n, [0] * n
        self.turns = [[0] * self.n_scales for _ in self.ctas]
        self.flight = []  # (the CTAs it touches, its barrier, bytes)
        self.commits = []  # in order: barriers
        self.synced = [0] * n
        self.give_up = give_up  # (role, the wait of it that gives up)
        self.errors, self.ended = [], set()
        self.drained = False

    # ------------------------------------------------------------ the roles; yield (barrier, parity) is a wait
    def codes(self, c):
        own_ok = True
        for s in range(self.total):
            own_ok = yield self.empty[c][s % self.n_codes], (s // self.n_codes - 1) & 1
            if not own_ok:
                break
            bar = self.full[0][s % self.n_codes]
            if c == 0:
                bar.arrive(BYTES * len(self.ctas))
            self.flight.append(((0, c), bar, BYTES))
            self.issued[c] += 1
        if self.rule == "own waits" and not self.pair and not own_ok:
            yield from self.drain_codes(self.issued[c])

    def scales(self, c):
        own_ok = True
        for s in range(self.total):
            own_ok = yield self.sempty[c][s % self.n_scales], (s // self.n_scales - 1) & 1
            if not own_ok:
                break
            bar = self.sfull[c][s % self.n_scales]
            bar.arrive(BYTES)
            self.flight.append(((c,), bar, BYTES))
            self.loaded[c] += 1
        if self.rule == "own waits" and not own_ok:
            yield from self.drain_scales(c)

    def turner(self, c, w):
        for i0 in range(0, self.total, self.n_scales):
            for slot in range(w, self.n_scales, self.turners):
                if i0 + slot >= self.total:
                    break
                if not (yield self.sfull[c][slot], (i0 // self.n_scales) & 1):
                    return
                if c == 0:
                    self.turned[0][slot].arrive(SIGNAL if self.pair else 0)
                else:
                    self.flight.append(((0, 1), self.turned[0][slot], SIGNAL))
                self.turns[c][slot] += 1

    def mma(self):
        s, ok = 0, True
        for t, stages in enumerate(self.tiles):
            ok = ok and (yield self.acce[0][t % 2], (t // 2 - 1) & 1)
            for kb in range(stages if ok else 0):
                ok = yield self.turned[0][s % self.n_scales], (s // self.n_scales) & 1
                ok = ok and (yield self.full[0][s % self.n_codes], (s // self.n_codes) & 1)
                if not ok:
                    break
                self.commits.append([self.sempty[c][s % self.n_scales] for c in self.ctas])
                self.commits.append([self.empty[c][s % self.n_codes] for c in self.ctas])
                if kb == stages - 1:
                    self.commits.append([self.accf[c][t % 2] for c in self.ctas])
                s += 1
        self.commits.append(self.finished)
        yield self.finished[0], 0, "drain"

    def epilogue(self, c):
        for t in range(len(self.tiles)):
            if not (yield self.accf[c][t % 2], (t // 2) & 1):
                return
            self.acce[0][t % 2].arrive()

    # ------------------------------------------------------------ the end of a CTA
    def drain_codes(self, issued):
        for i in range(max(0, issued - self.n_codes), issued):
            yield self.full[0][i % self.n_codes], (i // self.n_codes) & 1, "drain"

    def drain_scales(self, c):
        for i in range(max(0, self.loaded[c] - self.n_scales), self.loaded[c]):
            yield self.sfull[c][i % self.n_scales], (i // self.n_scales) & 1, "drain"

    def settle_codes(self):
        armed, issued = self.issued[0], self.issued[1]
        for i in range(max(0, max(armed, issued) - self.n_codes), max(armed, issued)):
            bar = self.full[0][i % self.n_codes]
            if i >= armed:
                bar.arrive(BYTES)
            elif i >= issued:
                bar.change(-BYTES)
            yield bar, (i // self.n_codes) & 1, "drain"

    def settle_signals(self):
        for slot in range(self.n_scales):
            mine, theirs = self.turns[0][slot], self.turns[1][slot]
            if theirs > mine:
                if theirs > mine + 1:
                    self.errors.append("a signal two turns ahead")
                self.turned[0][slot].arrive(SIGNAL)
            if theirs > 0:
                yield self.turned[0][slot], (theirs - 1) & 1, "drain"

    def end(self, c):
        gave_up = self.abort[c]
        if gave_up and self.rule == "all":
            yield from self.drain_scales(c)
            if not self.pair:
                yield from self.drain_codes(self.issued[c])
        if self.pair:
            if c == 0 and gave_up:
                self.abort[1] = self.unwind[1] = True
            yield from self.sync(c)
            if gave_up if c == 0 else self.unwind[1]:
                if c == 0:
                    yield from self.settle_codes()
                    if self.rule == "all":
                        yield from self.settle_signals()
                yield from self.sync(c)
        if any(c in touches for touches, _, _ in self.flight):
            self.errors.append("a copy in flight")
        if self.commits and c == 0:
            self.errors.append("a commit in flight")

    def sync(self, c):
        self.synced[c] += 1
        want = self.synced[c]
        yield lambda: min(self.synced) >= want

    # ------------------------------------------------------------ the schedule
    def run(self):
        roles = {}
        for c in self.ctas:
            roles[c, "codes"], roles[c, "scales"] = self.codes(c), self.scales(c)
            for w in range(self.turners):
                roles[c, f"turner{w}"] = self.turner(c, w)
            for w in range(2):
                roles[c, f"epilogue{w}"] = self.epilogue(c)
        roles[0, "mma"] = self.mma()
        speed = {k: self.rng.choice((0.05, 0.3, 1.0, 3.0)) for k in roles}
        landing = {n: self.rng.choice((0.002, 0.1, 0.5)) for n in (BYTES, SIGNAL)}
        seen = dict.fromkeys(roles, 0)
        asks = {}

        def step(k, *answer):
            try:
                asks[k] = roles[k].send(answer[0]) if answer else next(roles[k])
            except StopIteration:
                del roles[k]
                asks.pop(k, None)
                c = k[0]
                if k[1] == "end":
                    self.ended.add(c)
                elif not any(r[0] == c for r in roles):  # __syncthreads
                    roles[c, "end"], speed[c, "end"], seen[c, "end"] = self.end(c), 1.0, 0
                    step((c, "end"))

        def fail(k):
            if len(asks[k]) > 2:
                self.errors.append(f"{k}: a drain ran out")
            else:
                self.abort[k[0]] = True
            step(k, False)

        for k in list(roles):
            step(k)
        while roles:
            can = []
            for k, ask in asks.items():
                if callable(ask):
                    if ask():
                        can.append(("pass", k, speed[k]))
                elif ask[0].ready(ask[1]):
                    can.append(("pass", k, speed[k]))
                elif len(ask) == 2 and self.abort[k[0]]:
                    can.append(("fail", k, speed[k]))
            can += [("land", i, landing[n]) for i, (_, _, n) in enumerate(self.flight)]
            if self.commits:
                can.append(("commit", 0, 0.5))
            if not can:
                stuck = [k for k, ask in asks.items() if not callable(ask)]
                if not stuck:
                    self.errors.append("deadlock")
                    return self.errors
                fail(self.rng.choice(stuck))
                continue
            kind, k, _ = self.rng.choices(can, [x[2] for x in can])[0]
            if kind == "land":
                _, bar, n = self.flight.pop(k)
                bar.change(-n)
            elif kind == "commit":
                for bar in self.commits.pop(0):
                    bar.arrive()
            elif kind == "fail":
                step(k, False)
            elif callable(asks[k]) or len(asks[k]) > 2:
                step(k, True)
            else:
                seen[k] += 1
                if (k, seen[k]) == self.give_up:
                    fail(k)
                else:
                    step(k, True)
        return self.errors


def attempts(pair, rule, seeds):
    """A role and a wait of it that gives up, for each seed."""
    names = ["codes", "scales", "mma", "epilogue0", "epilogue1"] + [f"turner{w}" for w in range(depths(pair)[2])]
    for seed in seeds:
        rng = random.Random(1000 + seed)
        c = rng.randrange(2 if pair else 1)
        name = rng.choice(names)
        k = (0, name) if name == "mma" else (c, name)
        yield seed, k, Cluster(tiles(seed, 6), pair, seed, (k, rng.randint(1, 25)), rule).run()


@pytest.mark.parametrize("pair", [False, True])
def test_nothing_is_in_flight_when_a_cta_ends(pair):
    for seed, k, errors in attempts(pair, "all", range(250)):
        assert not errors, (pair, seed, k, errors[:3])


@pytest.mark.parametrize("pair", [False, True])
def test_a_call_in_which_no_wait_gives_up_ends_the_same_way(pair):
    for seed in range(25):
        for rule in ("all", "own waits"):
            cluster = Cluster(tiles(seed, 6), pair, seed, None, rule)
            assert not cluster.run() and not any(cluster.abort) and not any(cluster.unwind)


@pytest.mark.parametrize("pair", [False, True])
def test_draining_only_where_ones_own_wait_gave_up_leaves_copies_in_flight(pair):
    """A control: a warp whose copies were all issued before another role gave up does not wait for them,
    and nobody for the follower's signals."""
    assert any("a copy in flight" in errors for _, _, errors in attempts(pair, "own waits", range(250)))


def test_the_kernel_drains_after_its_roles_have_ended():
    """Where the kernel has its drains: behind the barrier that ends the roles, asked for by the CTA's flag."""
    from test_fp4_pipeline_cpu import SOURCE

    at = SOURCE.index("const bool gave_up = *abort_flag != 0u;")
    roles, end = SOURCE[:at], SOURCE[at:]
    assert "__syncthreads();" in roles[-500:]
    for bar in ("sfull_bar", "full_bar", "turned_bar"):
        assert f"drain_bar({bar}" not in roles and f"drain_bar({bar}" in end
    assert "pair_settle<kStages>" in end and "pair_report" not in SOURCE
