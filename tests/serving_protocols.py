"""Random-interleaving models of the barrier protocols of the decoding passes
over a cache (test infrastructure; see protocol_models.py for the method).

run_own: fa_serve_own.cuh (producer, MMA thread, softmax warps, one ring of K
and V tiles).  run_prefix: fa_tc_prefix.cu (producer, MMA thread, two softmax
slots).  Roles are generators that yield at every poll of a wait; loads land
and products complete at random times, the tensor pipe in issue order.  A run
fails if a barrier gets an arrival too many, a product reads a buffer with
other contents, a buffer is overwritten while a pending product reads it, or
a role waits for a phase that never comes.  `skip` names waits to leave out,
to show that the checks notice.
"""
import random

from protocol_models import Bar


class Machine:
    """Loads in flight, the tensor pipe, and what pending products read."""

    def __init__(self, rng):
        self.rng, self.loads, self.pipe, self.reads, self.has = rng, [], [], {}, {}

    def load(self, key, value, bar):
        self.loads.append((key, value, bar))

    def write(self, key, value):
        assert self.reads.get(key, 0) == 0, f"{key} = {value} over a buffer that a pending product reads"
        self.has[key] = value

    def product(self, reads, effect=None):
        """reads: {buffer: what it has to hold}; effect runs when the product is complete."""
        for k in reads:
            self.reads[k] = self.reads.get(k, 0) + 1
        self.pipe.append((reads, effect))

    def commit(self, bar):
        self.pipe.append((None, bar.arrive))

    def step(self):
        if self.loads and self.rng.random() < 0.5:
            key, value, bar = self.loads.pop(self.rng.randrange(len(self.loads)))
            self.write(key, value)
            bar.complete_tx(1)
            return True
        if self.pipe:
            reads, effect = self.pipe.pop(0)
            for k, v in (reads or {}).items():
                assert self.has.get(k) == v, f"product reads {k} = {self.has.get(k)}, not {v}"
                self.reads[k] -= 1
            if effect:
                effect()
            return True
        return bool(self.loads)


class Rendezvous:
    """A named barrier among n warps (the caller yields until it is past)."""

    def __init__(self, n):
        self.n, self.at, self.gen = n, 0, 0

    def come(self):
        gen = self.gen
        self.at += 1
        if self.at == self.n:
            self.at, self.gen = 0, self.gen + 1
        while self.gen == gen:
            yield


def drive(rng, roles, machine, limit=400000):
    speed = {r: 10 ** rng.uniform(-2, 0) for r in roles}
    engine = 10 ** rng.uniform(-2, 0)
    live = dict(roles)
    idle = 0
    for _ in range(limit):
        if not live:
            break
        names = list(live) + ["engine"]
        pick = rng.choices(names, [speed[n] if n != "engine" else engine for n in names])[0]
        if pick == "engine":
            machine.step()
            continue
        try:
            next(live[pick])
        except StopIteration:
            del live[pick]
    assert not live, f"roles that never finished: {sorted(live)}"
    while machine.step():
        pass


def wait(bar, parity):
    while not bar.try_wait(parity & 1):
        yield


def run_own(runs, seed, H=3, W=3, skip=()):
    """runs: tiles of each run; H ring slots; W softmax warps."""
    rng = random.Random(seed)
    m = Machine(rng)
    full, free = [Bar(f"full{i}", 1) for i in range(H)], [Bar(f"free{i}", 1) for i in range(H)]
    s = [Bar(f"s{i}", 1) for i in range(2)]
    p, o, q = [Bar(f"p{i}", W) for i in range(2)], [Bar(f"o{i}", 1) for i in range(2)], Bar("q", W)
    meet = Rendezvous(W)
    # runs whose first P V overwrote O^T; runs read out by every warp; steps added
    state = {"o": 0, "read": 0, "added": 0}
    outgrown = [rng.random() < 0.4 for _ in range(sum(runs))]  # steps that are weighed again

    def maybe(name, gen):
        if name not in skip:
            yield from gen

    def producer():
        h = 0
        for n in runs:
            for _ in range(2 * n):
                if h >= H:
                    yield from maybe("free", wait(free[h % H], h // H - 1))
                full[h % H].arrive(tx=1)
                m.load(("ring", h % H), h, full[h % H])
                h += 1
                yield

    def mma():
        g = 0

        def add(x, run, acc):
            h = 2 * x + 1
            yield from wait(full[h % H], h // H)
            yield from maybe("p", wait(p[x & 1], x >> 1))

            def effect():
                state["added"] += 1
                if not acc:
                    assert state["read"] == run * W, "O^T overwritten before it was read out"
                    state["o"] = run + 1

            m.product({("ring", h % H): h, **{("P", x & 1, w): x for w in range(W)}}, effect)
            m.commit(free[h % H])
            m.commit(o[x & 1])

        for run, n in enumerate(runs):
            yield from maybe("q", wait(q, run))
            for i in range(n):
                h = 2 * g
                yield from wait(full[h % H], h // H)

                def effect(x=g):
                    for w in range(W):
                        m.write(("S", x & 1, w), x)

                m.product({("ring", h % H): h, **{("Q", w): run for w in range(W)}}, effect)
                m.commit(free[h % H])
                m.commit(s[g & 1])
                if i > 0:
                    yield from add(g - 1, run, i > 1)
                g += 1
                yield
            yield from add(g - 1, run, n > 1)

    def softmax(w):
        def put_q(run):
            m.write(("Q", w), run)
            yield from meet.come()
            q.arrive()

        g = 0
        yield from put_q(0)
        for run, n in enumerate(runs):
            for i in range(n):
                yield from maybe("s", wait(s[g & 1], g >> 1))
                assert m.has.get(("S", g & 1, w)) == g, "scores of another step"
                yield
                if i == 0:  # references, then the weights
                    yield from meet.come()
                    yield from meet.come()
                for again in range(1 + (i > 0 and outgrown[g])):
                    assert m.has.get(("S", g & 1, w)) == g, "scores overwritten while in use"
                    m.write(("P", g & 1, w), g)
                    yield
                    if i > 0 and not again:
                        yield from meet.come()  # the vote
                        if outgrown[g]:  # references, O^T rescaled, and once more
                            yield from maybe("o", wait(o[(g - 1) & 1], (g - 1) >> 1))
                            yield from meet.come()
                            yield from meet.come()
                            assert state["added"] == g, "O^T rescaled while steps are missing"
                p[g & 1].arrive()
                g += 1
            yield from meet.come()
            if run + 1 < len(runs):
                yield from put_q(run + 1)
            yield from maybe("o_end", wait(o[(g - 1) & 1], (g - 1) >> 1))
            yield from meet.come()
            assert state["o"] == run + 1, "state read before the run's products"
            state["read"] += 1
            yield from meet.come()

    drive(rng, {"producer": producer(), "mma": mma(), **{f"w{w}": softmax(w) for w in range(W)}}, m)


def run_prefix(runs, seed, S=2, W=2, skip=(), one_barrier=False, scrub=False, scrub_slot=0):
    """runs: (steps, slots) of each run; S stages; W softmax warps a slot.
    one_barrier: a run's last P V announced on the barrier of the scores.
    scrub: the warps of scrub_slot write into V before they announce their weights, at some steps."""
    rng = random.Random(seed)
    m = Machine(rng)
    k0, kv = Bar("k0", 1), [Bar(f"kv{i}", 1) for i in range(S)]
    kfree, vfree = [Bar(f"kfree{i}", 1) for i in range(S)], [Bar(f"vfree{i}", 1) for i in range(S)]
    bq, bs = [Bar(f"q{t}", W) for t in range(2)], [Bar(f"s{t}", 1) for t in range(2)]
    bp, fin = [Bar(f"p{t}", W) for t in range(2)], [Bar(f"fin{t}", 1) for t in range(2)]
    total = sum(n for n, _ in runs)
    starts = [sum(n for n, _ in runs[:i]) for i in range(len(runs))]
    read = {(t, r): 0 for t in range(2) for r in range(len(runs))}
    complete = set()  # (slot, run) whose last P V is done
    scrubbed = [scrub and rng.random() < 0.5 for _ in range(total)]

    def maybe(name, gen):
        if name not in skip:
            yield from gen

    def producer():
        k0.arrive(tx=1)
        m.load(("K", 0), 0, k0)
        for g in range(total):
            if g >= S:
                yield from maybe("vfree", wait(vfree[g % S], g // S - 1))
            if g + 1 < total and g + 1 >= S:
                yield from maybe("kfree", wait(kfree[(g + 1) % S], (g + 1) // S - 1))
            kv[g % S].arrive(tx=2 if g + 1 < total else 1)
            m.load(("V", g % S), g, kv[g % S])
            if g + 1 < total:
                m.load(("K", (g + 1) % S), g + 1, kv[g % S])
            yield

    def mma():
        cp, used = [0, 0], [0, 0]

        def scores(t, r, g):
            def effect():
                for w in range(W):
                    m.has[("SP", t, w)] = ("S", g)

            m.product({("K", g % S): g, **{("Q", t, w): r for w in range(W)}}, effect)

        yield from wait(k0, 0)
        for r, (n, slots) in enumerate(runs):
            G = starts[r]
            for t in range(slots):
                yield from maybe("q", wait(bq[t], used[t]))
                used[t] += 1
                scores(t, r, G)
                m.commit(bs[t])
            for j in range(n):
                g = G + j
                yield from wait(kv[g % S], g // S)
                for t in range(slots):
                    yield from maybe("p", wait(bp[t], cp[t]))
                    cp[t] += 1

                    def effect(t=t, r=r, first=j == 0, last=j == n - 1):
                        before = [x for x in range(r) if runs[x][1] > t]
                        if first and before:
                            assert read[t, before[-1]] == W, "accumulator overwritten before it was read out"
                        if last:
                            complete.add((t, r))

                    m.product({("V", g % S): g, **{("SP", t, w): ("P", g) for w in range(W)}}, effect)
                    if j + 1 < n:
                        scores(t, r, g + 1)
                    m.commit(bs[t] if j + 1 < n or one_barrier else fin[t])
                    yield

    def softmax(t, w):
        mine = [r for r, (_, slots) in enumerate(runs) if t < slots]
        cs, f, ready = 0, 0, False
        for x, r in enumerate(mine):
            n, slots = runs[r]
            if not ready:
                m.write(("Q", t, w), r)
                bq[t].arrive()
            ready = False
            for j in range(n):
                g = starts[r] + j
                yield from maybe("s", wait(bs[t], cs))
                cs += 1
                if t == slots - 1 and w == 0:
                    kfree[g % S].arrive()
                    if g > 0:
                        vfree[(g - 1) % S].arrive()
                assert m.has.get(("SP", t, w)) == ("S", g), "scores of another step"
                yield
                m.write(("SP", t, w), ("P", g))
                yield
                if scrubbed[g] and t == min(scrub_slot, slots - 1):
                    yield from maybe("scrub", wait(kv[g % S], g // S))
                    assert m.has.get(("V", g % S)) == g, "values of another step"
                    m.write(("V", g % S), g)
                bp[t].arrive()
            if r + 1 < len(runs) and t < runs[r + 1][1]:
                m.write(("Q", t, w), r + 1)
                bq[t].arrive()
                ready = True
            if one_barrier:
                yield from wait(bs[t], cs)
                cs += 1
            else:
                yield from maybe("fin", wait(fin[t], f))
                f += 1
            assert (t, r) in complete, "state read before the run's products"
            read[t, r] += 1
            yield

    roles = {"producer": producer(), "mma": mma()}
    roles.update({f"s{t}{w}": softmax(t, w) for t in range(2) for w in range(W)})
    drive(rng, roles, m)
