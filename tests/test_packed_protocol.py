"""Models of the mbarrier protocols of the packed attention's tensor-core
kernels, run on the CPU under schedules that hold single warps back.

Every role of a block (loading warps, warps that issue matrix products, softmax
warps) is a generator that waits and arrives as the kernel does.  Loads land in
any order.  A thread's matrix products run in the order in which it issued them,
those of two threads in any order, and a commit arrives once the thread's
products before it have run.  A parity wait succeeds when the current phase's
parity differs from the one waited for, as mbarrier.try_wait.parity does: a
warp that comes to a barrier two phases late finds it as if nothing had
happened, and waits for good.  The scheduler runs roles by priorities that it
changes at random, so that any warp may sleep while the others go as far as
they can.

Checked are that nothing deadlocks, that every wait that passes has seen the
phase it was meant for, and that every product and every softmax finds the
tiles it was meant for.  How many barriers stand for a step's S, dS and turn is
read from the sources.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "vision_sliding_window_b200", "csrc")


def barriers_of(name):
    """How many barriers the kernels of na_packed_tc_bwd.cu use in turn for a step's `name`."""
    with open(os.path.join(CSRC, "na_packed_tc_bwd.cu")) as f:
        source = f.read()
    two = re.search(rf"uint32_t {name}\(int i\) const {{ return base \+ \d+ \+ \(i & 1\) \* 8; }}", source)
    # every wait for it looks for the phase that goes with that
    waits = set(re.findall(rf"mbar_wait\([^;]*?bar\.{name}\((\w*)\)(?: : bar\.\w+\(i\))?, ([^,]*), ab", source))
    assert waits == ({("i", "(i >> 1) & 1")} if two else {("", "i & 1")}), (name, waits)
    return 2 if two else 1


class Stuck(AssertionError):
    pass


class Barrier:
    def __init__(self, name, count=1):
        self.name, self.count, self.done, self.pending = name, count, 0, 0

    def arrive(self):
        self.pending += 1
        if self.pending == self.count:
            self.pending, self.done = 0, self.done + 1

    def passed(self, phase):
        ok = (self.done & 1) != (phase & 1)
        if ok and self.done != phase + 1:
            raise Stuck(f"{self.name}: a wait for phase {phase} passed with {self.done} complete")
        return ok


class InTurn:
    """`slots` barriers for the steps 0, 1, 2, ..."""

    def __init__(self, name, slots, count=1):
        self.slots = [Barrier(f"{name}{i}", count) for i in range(slots)]

    def arrive(self, i):
        self.slots[i % len(self.slots)].arrive()

    def wait(self, i):
        bar = self.slots[i % len(self.slots)]
        while not bar.passed(i // len(self.slots)):
            yield False


class Block:
    def __init__(self, seed):
        self.rnd = random.Random(seed)
        self.roles, self.loads, self.pipes = [], [], {}

    def role(self, name, gen):
        self.roles.append([self.rnd.random(), name, gen])

    def load(self, land):
        self.loads.append(land)

    def issue(self, thread, op):  # a product or a commit
        self.pipes.setdefault(thread, []).append(op)

    def fire(self):
        """Lets one load land or one thread's next product run."""
        ready = [("load", i) for i in range(len(self.loads))] + [("pipe", t) for t, ops in self.pipes.items() if ops]
        if not ready:
            return False
        kind, which = self.rnd.choice(ready)
        (self.loads.pop(which) if kind == "load" else self.pipes[which].pop(0))()
        return True

    def run(self):
        hardware, idle = self.rnd.random(), 0
        while self.roles:
            if self.rnd.random() < 0.05:  # someone falls asleep or wakes
                self.rnd.choice(self.roles)[0] = self.rnd.random()
            if self.rnd.random() < 0.05:
                hardware = self.rnd.random()
            self.roles.sort(key=lambda r: -r[0])
            fired = False
            for r in list(self.roles):
                if not fired and hardware > r[0]:
                    fired = True
                    if self.fire():
                        break
                try:
                    if next(r[2]):
                        break
                except StopIteration:
                    self.roles.remove(r)
                    break
            else:
                # a role that came to its next wait has perhaps let an earlier one go on
                idle = 0 if self.fire() else idle + 1
                if idle > len(self.roles) + 1:
                    raise Stuck("deadlock: " + ", ".join(r[1] for r in self.roles))
                continue
            idle = 0
        while self.fire():
            pass


def expect(have, want, what):
    if have != want:
        raise Stuck(f"{what}: found {have}, wanted {want}")


WARPS = 2  # softmax warps (eight in the kernel)


def rings(block, n, sa, sb, empty_b, tail):
    """The two loading warps' rings, with their last tile's barrier."""
    full_a, empty_a = InTurn("full_a", sa), InTurn("empty_a", sa)
    full_b, empty_b = InTurn("full_b", sb), InTurn("empty_b", sb, empty_b)
    both, a, b = Barrier("tail", 2), [None] * sa, [None] * sb

    def loader(slots, full, empty, tiles, before):
        for i in range(n):
            yield from before(i)
            if i >= slots:
                yield from empty.wait(i - slots)
            cut = tail and i == n - 1

            def land(i=i, cut=cut):
                tiles[i % slots] = i
                both.arrive() if cut else full.arrive(i)
            block.load(land)
            yield True
            if cut:
                while not both.passed(0):
                    yield False
                full.arrive(i)

    return full_a, empty_a, full_b, empty_b, a, b, loader


def no_wait(i):
    return
    yield


def dq(n, seed, sa, sb, tail, s_slots, dp_slots, ds_slots, turn_slots):
    block = Block(seed)
    full_a, empty_a, full_b, empty_b, k, v, loader = rings(block, n, sa, sb, 1, tail)
    kept = Barrier("kept")
    s, dp = InTurn("s", s_slots), InTurn("dp", dp_slots)
    ds_ready, turn = InTurn("ds_ready", ds_slots, WARPS), InTurn("turn", turn_slots)
    S, dP, dQ = [None, None], [None], [0]
    read = [[0] * WARPS, [0] * WARPS]  # steps whose S and dP a warp has read

    def stays():
        block.load(kept.arrive)
        yield True

    def make(thread, tiles, i, slots, to, at, holds, commits):
        def product():
            expect(tiles[i % slots], i, f"{thread}'s tile")
            expect(holds(), True, f"{thread} writes over step {i}")
            to[at] = i
        block.issue(thread, product)
        for c in commits:
            block.issue(thread, c)

    def s_free(i):  # S of step i - 2 and its dS have been used
        return lambda: i < 2 or (dQ[0] >= i - 1 and min(read[0]) >= i - 1)

    def warp1():
        while not kept.passed(0):
            yield False
        yield from full_a.wait(0)
        make("S", k, 0, sa, S, 0, s_free(0), [lambda: s.arrive(0)])
        for i in range(n):
            if i + 1 < n:
                yield from full_a.wait(i + 1)
                make("S", k, i + 1, sa, S, (i + 1) & 1, s_free(i + 1), [lambda i=i: s.arrive(i + 1)])
                yield True
            yield from ds_ready.wait(i)
            yield from turn.wait(i)

            def add(i=i):
                expect(k[i % sa], i, "dQ's keys")
                expect(S[i & 1], ("dS", i), "dQ's weights")
                dQ[0] += 1
            block.issue("S", add)
            block.issue("S", lambda i=i: empty_a.arrive(i))
            yield True

    def warp2():
        while not kept.passed(0):
            yield False
        yield from full_b.wait(0)

        def product(i):
            make("dP", v, i, sb, dP, 0, lambda: min(read[1]) >= i,
                 [lambda: dp.arrive(i), lambda: empty_b.arrive(i)])
        product(0)
        for i in range(n):
            yield from ds_ready.wait(i)
            if i + 1 < n:
                yield from full_b.wait(i + 1)
                product(i + 1)
            yield True
            turn.arrive(i)

    written = {}

    def softmax(w):
        yield True
        for i in range(n):
            yield from s.wait(i)
            expect(S[i & 1], i, "softmax's S")
            yield True
            yield from dp.wait(i)
            expect(dP[0], i, "softmax's dP")
            read[0][w] = read[1][w] = i + 1
            yield True
            written[i] = written.get(i, 0) + 1
            if written[i] == WARPS:
                S[i & 1] = ("dS", i)
            ds_ready.arrive(i)

    block.role("stays", stays())
    block.role("loader a", loader(sa, full_a, empty_a, k, no_wait))
    block.role("loader b", loader(sb, full_b, empty_b, v, no_wait))
    block.role("warp 1", warp1())
    block.role("warp 2", warp2())
    for w in range(WARPS):
        block.role(f"softmax {w}", softmax(w))
    block.run()
    expect(dQ[0], n, "steps summed")


def dkdv(n, seed, sa, sb, tail, s_slots, dp_slots, half_slots, p_slots, ds_slots, turn_slots):
    block = Block(seed)
    full_a, empty_a, full_b, empty_b, q, o, loader = rings(block, n, sa, sb, 2, tail)
    full_t, empty_t, terms = InTurn("full_t", 2), InTurn("empty_t", 2, WARPS), [None, None]
    kept, s, dp = Barrier("kept"), InTurn("s", s_slots), InTurn("dp", dp_slots)
    p_half, p_ready = InTurn("p_half", half_slots, WARPS), InTurn("p_ready", p_slots, WARPS)
    ds_ready = InTurn("ds_ready", ds_slots, WARPS)
    turn = InTurn("turn", turn_slots)
    S, dP, sums = [None], [None], [0, 0]

    def stays():
        block.load(kept.arrive)
        yield True

    def load_terms(i):
        if i >= 2:
            yield from empty_t.wait(i - 2)
        terms[i % 2] = i
        full_t.arrive(i)

    def make(thread, tiles, i, slots, to, before, commits):
        def product():
            expect(tiles[i % slots], i, f"{thread}'s tile")
            expect(to[0] if i else before, before, f"{thread} writes over step {i}")
            to[0] = i
        block.issue(thread, product)
        for c in commits:
            block.issue(thread, c)

    def add(thread, which, weights, i, tiles, slots, what):
        def product():
            expect(tiles[i % slots], i, f"{what}'s tile")
            expect(weights[0], (what, i), f"{what}'s weights")
            sums[which] += 1
        block.issue(thread, product)

    def warp1():
        while not kept.passed(0):
            yield False
        yield from full_a.wait(0)
        make("one", q, 0, sa, S, None, [lambda: s.arrive(0)])
        for i in range(n):
            yield from full_b.wait(i)
            if i + 1 < n:
                yield from full_a.wait(i + 1)
            yield from p_half.wait(i)
            yield True
            yield from p_ready.wait(i)
            add("one", 0, S, i, o, sb, "P")
            block.issue("one", lambda i=i: empty_b.arrive(i))
            if i + 1 < n:
                make("one", q, i + 1, sa, S, ("P", i), [lambda i=i: s.arrive(i + 1)])
            yield True
            turn.arrive(i)

    def warp3():
        while not kept.passed(0):
            yield False
        yield from full_b.wait(0)

        def product(i):
            make("two", o, i, sb, dP, ("dS", i - 1), [lambda: dp.arrive(i), lambda: empty_b.arrive(i)])
        product(0)
        for i in range(n):
            yield from full_a.wait(i)
            if i + 1 < n:
                yield from full_b.wait(i + 1)
            yield from ds_ready.wait(i)
            yield from turn.wait(i)
            add("two", 1, dP, i, q, sa, "dS")
            block.issue("two", lambda i=i: empty_a.arrive(i))
            if i + 1 < n:
                product(i + 1)
            yield True

    counts = {}

    def all_of(key):
        counts[key] = counts.get(key, 0) + 1
        return counts[key] == WARPS

    def softmax(w):
        for i in range(n):
            yield from full_t.wait(i)
            yield from s.wait(i)
            expect(terms[i % 2], i, "softmax's terms")
            expect(S[0] in (i, ("P", i)), True, "softmax's S")
            yield True
            p_half.arrive(i)
            yield True
            if all_of(("P", i)):
                S[0] = ("P", i)
            p_ready.arrive(i)
            yield from dp.wait(i)
            expect(dP[0], i, "softmax's dP")
            expect(terms[i % 2], i, "softmax's terms")
            yield True
            if all_of(("dS", i)):
                dP[0] = ("dS", i)
            ds_ready.arrive(i)
            empty_t.arrive(i)

    block.role("stays", stays())
    block.role("loader a", loader(sa, full_a, empty_a, q, no_wait))
    block.role("loader b", loader(sb, full_b, empty_b, o, load_terms))
    block.role("warp 1", warp1())
    block.role("warp 3", warp3())
    for w in range(WARPS):
        block.role(f"softmax {w}", softmax(w))
    block.run()
    expect(sums, [n, n], "steps summed")


def forward(steps, seed, slots=4):
    """The forward: a row tile for each of `steps`, which counts its key tiles; one
    S that the tiles use in turn, a ring of K_0, V_0, K_1, V_1, ..."""
    block, n = Block(seed), max(steps)
    full, empty = InTurn("full", slots), InTurn("empty", slots)
    s, pv = [InTurn("s", 1) for _ in steps], [InTurn("pv", 1) for _ in steps]
    p = [[InTurn("p", 1, WARPS) for _ in range(2)] for _ in steps]
    free, kept = InTurn("free", 1, WARPS), Barrier("q")
    ring, S, readers = [None] * slots, [None], [0]
    P, O, written = [[None, None] for _ in steps], [0 for _ in steps], {}

    def loader():
        block.load(kept.arrive)
        for i in range(2 * n):
            if i >= slots:
                yield from empty.wait(i - slots)

            def land(i=i):
                ring[i % slots] = i
                full.arrive(i)
            block.load(land)
            yield True

    def products_s():
        while not kept.passed(0):
            yield False
        made = 0
        for j in range(n):
            yield from full.wait(2 * j)
            for t, k in enumerate(steps):
                if j >= k:
                    continue
                if made:
                    yield from free.wait(made - 1)
                made += 1

                def product(t=t, j=j):
                    expect(ring[2 * j % slots], 2 * j, "S's keys")
                    expect(readers[0], 0, "warps that still read S")
                    S[0], readers[0] = (t, j), WARPS
                block.issue("S", product)
                block.issue("S", lambda t=t, j=j: s[t].arrive(j))
                yield True
            block.issue("S", lambda j=j: empty.arrive(2 * j))

    def products_pv():
        for j in range(n):
            yield from full.wait(2 * j + 1)
            for t, k in enumerate(steps):
                if j >= k:
                    continue
                for half in range(2):
                    yield from p[t][half].wait(j)

                    def product(t=t, j=j, half=half):
                        expect(ring[(2 * j + 1) % slots], 2 * j + 1, "the values")
                        expect(P[t][half], j, "the weights")
                        O[t] += half
                    block.issue("PV", product)
                    yield True
                block.issue("PV", lambda t=t, j=j: pv[t].arrive(j))
            block.issue("PV", lambda j=j: empty.arrive(2 * j + 1))

    def softmax(t, w):
        for j in range(steps[t]):
            yield from s[t].wait(j)
            expect(S[0], (t, j), "softmax's S")
            yield True
            readers[0] -= 1
            free.arrive(0)
            if j:
                yield from pv[t].wait(j - 1)
                expect(O[t], j, "products before O is rescaled")
            for half in range(2):
                yield True
                written[t, j, half] = written.get((t, j, half), 0) + 1
                if written[t, j, half] == WARPS:
                    P[t][half] = j
                p[t][half].arrive(j)
        if steps[t]:
            yield from pv[t].wait(steps[t] - 1)
            expect(O[t], steps[t], "products at the end")

    block.role("loader", loader())
    block.role("S", products_s())
    block.role("PV", products_pv())
    for t in range(len(steps)):
        for w in range(WARPS):
            block.role(f"softmax {t} {w}", softmax(t, w))
    block.run()


def few_rows(tiles, seed, slots):
    """The kernel for few rows: row tiles of `tiles` key tiles each go through one
    ring; all warps meet between them, as the join's sums take the ring's place."""
    block = Block(seed)
    full, empty = InTurn("full", slots), InTurn("empty", slots, WARPS)
    ring, met, reading = [None] * slots, [0], [0]

    def meet(k):
        met[0] += 1
        while met[0] < k * (WARPS + 1):
            yield False

    def loader():
        done = 0
        for k, n in enumerate(tiles):
            for u in range(done, done + n):
                if u >= slots:
                    yield from empty.wait(u - slots)

                def land(u=u):
                    expect(ring[u % slots] in ("sums", None, u - slots), True, "a slot that is loaded over")
                    ring[u % slots] = u
                    full.arrive(u)
                block.load(land)
                yield True
            for u in range(max(done, done + n - slots), done + n):  # settles
                yield from full.wait(u)
            done += n
            yield from meet(2 * k + 1)
            yield from meet(2 * k + 2)

    def warp(w):
        done = 0
        for k, n in enumerate(tiles):
            for u in range(done, done + n):
                yield from full.wait(u)
                expect(ring[u % slots], u, "a warp's tile")
                yield True
                empty.arrive(u)
            done += n
            reading[0] += 1
            while reading[0] < (k + 1) * WARPS:  # all warps have read the ring
                yield False
            expect(block.loads, [], "copies in flight over the sums")
            for i in range(slots):
                ring[i] = "sums"
            yield from meet(2 * k + 1)
            expect(set(ring), {"sums"}, "the sums when they are read")
            yield True
            yield from meet(2 * k + 2)

    block.role("loader", loader())
    for w in range(WARPS):
        block.role(f"warp {w}", warp(w))
    block.run()


@pytest.mark.parametrize("steps", [(1,), (2,), (7,), (1, 1), (1, 2), (5, 5), (5, 6), (0, 3), (4, 0)])
def test_forward(steps):
    for seed in range(150):
        forward(steps, seed)


@pytest.mark.parametrize("slots", [1, 3, 8])
@pytest.mark.parametrize("tiles", [(1,), (9,), (3, 0, 5), (1, 2, 3, 4), (0, 0, 2), (20, 20)])
def test_few_rows(tiles, slots):
    for seed in range(100):
        few_rows(tiles, seed, slots)


RINGS = [(3, 2), (4, 4)]  # slots of the two rings at d = 128 and below
SEEDS = range(60)
OF_DQ = ("s", "dp", "ds_ready", "turn")
OF_DKDV = ("s", "dp", "p_half", "p_ready", "ds_ready", "turn")


@pytest.mark.parametrize("sa,sb", RINGS)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("kernel,names", [(dq, OF_DQ), (dkdv, OF_DKDV)])
def test_no_warp_is_overrun(kernel, names, sa, sb, tail):
    slots = [barriers_of(name) for name in names]
    for n in (1, 2, 3, 5, 9):
        for seed in SEEDS:
            kernel(n, seed, sa, sb, tail, *slots)


@pytest.mark.parametrize("kernel,names,one", [(dq, OF_DQ, "s"), (dq, OF_DQ, "ds_ready"), (dq, OF_DQ, "turn"),
                                              (dkdv, OF_DKDV, "turn")])
def test_one_barrier_for_all_steps_can_be_overrun(kernel, names, one):
    with pytest.raises(Stuck):
        for n in (3, 5, 9):
            for seed in range(400):
                kernel(n, seed, 4, 4, False, *(1 if name == one else 2 for name in names))


# ------------------------------------------------------------- waits given up
# A wait that runs out raises the block's flag and every other wait gives up
# too.  Copies that are in flight then must have landed before the block ends.
def source_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def given_up(slots, n, seed, settles):
    """A warp that loads n tiles into a ring, a warp that uses them, and a wait of
    either that runs out while the loads that are in flight are late."""
    rnd = random.Random(seed)
    full, empty = InTurn("full", slots), InTurn("empty", slots)
    loads, gave_up, at = [], [False], rnd.randint(0, 3 * n)

    def wait(bar, i):
        b = bar.slots[i % slots]
        while (b.done & 1) == ((i // slots) & 1):
            if gave_up[0]:
                return False
            yield
        return True

    def loader():
        asked = 0
        for i in range(n):
            if i >= slots and not (yield from wait(empty, i - slots)):
                break
            loads.append(i)
            asked += 1
            yield
        if settles:
            for u in range(max(0, asked - slots), asked):
                while u in loads:
                    yield

    def user():
        for i in range(n):
            if not (yield from wait(full, i)):
                break
            empty.arrive(i)
            yield

    roles, late = [loader(), user()], rnd.random()
    for step in range(10000):
        if step >= at:
            gave_up[0] = True
        if loads and rnd.random() > late:
            i = loads.pop(rnd.randrange(len(loads)))
            full.arrive(i)
        if roles:
            r = rnd.choice(roles)
            if next(r, "over") == "over":
                roles.remove(r)
        if not roles:
            if loads:
                raise Stuck(f"tiles {loads} in flight when the block ended")
            return
    raise Stuck("deadlock")


@pytest.mark.parametrize("kernel", ["na_packed_tc.cu", "na_packed_tc_bwd.cu", "na_packed_rows.cu", "na_norm.cu"])
def test_no_copy_is_in_flight_when_a_block_ends(kernel):
    source = source_of(kernel)
    if kernel == "na_norm.cu":  # the warp that asks settles before it leaves
        left = re.findall(r"if \(!__all_sync\(0xffffffffu, mbar_wait\([^;{]*\{\n\s*if \(threadIdx.x < 32\) ring_settle\(", source)
        settles = len(left) == source.count("mbar_wait(ring.bar(it)") == 2
    else:  # every loading warp settles, whether or not a wait was given up by then
        loops = len(re.findall(r"-- loads|- loads: ", source))
        settles = len(re.findall(r"\n      settle_ring\(", source)) == loops > 0
    for slots in (1, 2, 4, 8):
        for n in (1, 3, 9, 20):
            for seed in range(100):
                given_up(slots, n, seed, settles)


def test_a_loading_warp_that_leaves_at_once_is_found():
    with pytest.raises(Stuck, match="in flight"):
        for seed in range(100):
            given_up(4, 9, seed, False)
