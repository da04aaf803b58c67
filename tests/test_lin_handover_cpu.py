"""The hand-overs of the linear-attention prefill kernel (csrc/lin_prefill.cu) in a
model of its barriers: workers, row warp, product warp and factor warps as programs
of waits, arrivals and accesses, run in random orders.  A barrier's phase is known by
its parity alone, as on the GPU, so that a waiter that falls two phases behind hangs;
every access is checked for what it may not overlap."""
import random

import pytest

STAGES, BUFS, NORMS = 3, 4, 2


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def ready(self, phase):  # try_wait.parity: the phase of this parity is over
        return (self.phase & 1) != (phase & 1)


class Cta:
    """What the programs share: barriers, who holds what, and the order of products."""

    def __init__(self, nch, local, workers=3, pool=False):
        self.nch, self.local, self.workers, self.pool = nch, local, workers, pool
        self.bar = {("in", i): Barrier(NORMS) for i in range(BUFS)}
        self.bar |= {("gate", i): Barrier(1) for i in range(BUFS)}
        self.bar |= {(x, i): Barrier(1) for x in ("full", "empty") for i in range(STAGES)}
        self.bar |= {("free", i): Barrier(workers) for i in range(BUFS)}
        self.bar |= {("wk", i): Barrier(workers) for i in range(2)}
        self.bar |= {("ds", i): Barrier(1) for i in range(2)}
        self.bar |= {("u", 0): Barrier(workers), ("s", 0): Barrier(workers), ("s", 1): Barrier(workers), ("p", 0): Barrier(workers), ("qk", 0): Barrier(1), ("o", 0): Barrier(1)}
        self.bar |= {("state", 0): Barrier(1), ("read", 0): Barrier(1), ("met", 0): Barrier(workers)}
        # the pool's state lands where these will be
        self.state = [("wk", 1, x) for x in range(workers)] if local else [(x, 2) for x in ("K", "V", "Q")] + [
            ("P", x) for x in range(workers)]
        self.queue = []  # products and commits in issue order
        self.holds = {}  # resource -> chunk whose data it holds
        self.reading = {}  # resource -> products under way that read or write it

    def put(self, what, chunk):
        """Data of `chunk` goes into a place that no product under way uses."""
        assert not self.reading.get(what), f"{what} overwritten for chunk {chunk} under a product"
        self.holds[what] = chunk

    def use(self, what, chunk):
        assert self.holds.get(what) == chunk, f"{what} holds {self.holds.get(what)}, wanted {chunk}"

    def use_factors(self, chunk):
        self.use(("decays", chunk % BUFS), chunk)
        for i in range(NORMS):
            self.use(("factors", chunk % BUFS, i), chunk)

    def product(self, reads, writes, chunk):
        for r in reads:
            self.use(r, chunk)
        for x in list(reads) + list(writes):
            self.reading[x] = self.reading.get(x, 0) + 1
        for x in writes:
            self.holds[x] = None  # until it is done
        self.queue.append(("product", list(reads) + list(writes), list(writes), chunk))

    def commit(self, bar):
        self.queue.append(("commit", bar))

    def step_queue(self):
        kind, *x = self.queue.pop(0)
        if kind == "commit":
            self.bar[x[0]].arrive()
        else:
            for r in x[0]:
                self.reading[r] -= 1
            for w in x[1]:
                self.holds[w] = x[2]


def rows(t):
    for c in range(t.nch):
        if c >= STAGES:
            yield ("empty", c % STAGES), c // STAGES - 1
        if c == 2 and t.pool and not t.local:
            yield ("read", 0), 0
        for what in ("K", "V", "Q"):
            t.put((what, c % STAGES), c)
        yield
        t.bar["full", c % STAGES].arrive()
        if c == 0 and t.pool:
            for place in t.state:
                t.put(place, "state")
            yield
            t.bar["state", 0].arrive()
        yield


def factors(t, which):
    for c in range(which, t.nch, 2):
        if c >= BUFS:
            yield ("free", c % BUFS), c // BUFS - 1
        t.holds["decays", c % BUFS] = c
        yield
        t.bar["gate", c % BUFS].arrive()
        yield


def norms(t, i):
    for c in range(t.nch):
        yield ("full", c % STAGES), c // STAGES
        for what in ("K",) if t.local else ("K", "Q"):
            t.use((what, c % STAGES), c)
            yield
        t.use((what, c % STAGES), c)
        yield ("gate", c % BUFS), c // BUFS
        t.use(("decays", c % BUFS), c)
        t.holds["factors", c % BUFS, i] = c
        yield
        t.bar["in", c % BUFS].arrive()
        yield


def worker(t, w):
    """Worker w: its share of every place is a place of its own; a product needs all."""
    n = t.nch

    def keys(c):
        yield ("in", c % BUFS), c // BUFS
        t.use_factors(c)
        t.use(("K", c % STAGES), c)
        if w == 0:
            t.put(("V", c % STAGES), c)  # rows past the end zeroed
        t.put(("wk", c & 1 if t.local else 0, w), c)

    def update(c):
        t.use(("dS", c & 1 if t.local else 0), c)

    def outputs(c):
        t.use(("O1", c & 1), c)
        t.use(("O2", c & 1), c)
        t.use_factors(c)
        yield
        t.bar["free", c % BUFS].arrive()

    yield from keys(0)
    yield
    t.bar["wk", 0].arrive()
    if t.pool:
        yield ("state", 0), 0
        for place in t.state:
            t.use(place, "state")
            yield
        t.bar["met", 0].arrive()
        yield ("met", 0), 0
        if w == 0:
            t.bar["read", 0].arrive()
    for c in range(n):
        if t.local:
            if c > 0:
                yield ("ds", (c - 1) & 1), (c - 1) >> 1
                update(c - 1)
                yield
            t.use_factors(c)
            if c + 1 < n:
                yield from keys(c + 1)
                yield
                t.bar["wk", (c + 1) & 1].arrive()
            yield
            t.bar["free", c % BUFS].arrive()
            yield
        else:
            if c > 0:
                update(c - 1)
                yield
                update(c - 1)
            t.bar["u", 0].arrive()
            yield
            t.use_factors(c)
            yield
            t.put(("S", c & 1, w), c)
            yield
            t.bar["s", c & 1].arrive()
            yield ("qk", 0), c
            t.use(("QK", c & 1), c)
            t.use_factors(c)
            yield
            t.put(("P", w), c)
            yield
            t.bar["p", 0].arrive()
            yield
            if c > 0:
                yield from outputs(c - 1)
            yield ("ds", c & 1), c >> 1
            if c + 1 < n:
                yield from keys(c + 1)
                yield
                t.bar["wk", (c + 1) & 1].arrive()
            yield
    if t.local:
        yield ("ds", (n - 1) & 1), (n - 1) >> 1
    else:
        yield ("o", 0), 0
        yield from outputs(n - 1)
    update(n - 1)


def products(t):
    W = range(t.workers)
    for c in range(t.nch):
        st = c % STAGES
        yield ("in", c % BUFS), c // BUFS
        yield ("wk", c & 1), c >> 1
        wk = c & 1 if t.local else 0
        if t.local:
            t.product([("V", st)] + [("wk", wk, x) for x in W], [("dS", wk)], c)
            t.commit(("ds", c & 1))
            t.commit(("empty", st))
            yield
            continue
        t.product([("Q", st), ("K", st)], [("QK", c & 1)], c)
        t.commit(("qk", 0))
        yield ("u", 0), c
        t.product([("V", st)] + [("wk", 0, x) for x in W], [("dS", 0)], c)
        t.commit(("ds", c & 1))
        yield ("s", c & 1), c >> 1
        t.product([("Q", st)] + [("S", c & 1, x) for x in W], [("O1", c & 1)], c)
        yield ("p", 0), c
        t.product([("V", st)] + [("P", x) for x in W], [("O2", c & 1)], c)
        t.commit(("empty", st))
        if c == t.nch - 1:
            t.commit(("o", 0))
        yield


def run(nch, local, seed):
    rng = random.Random(seed)
    t = Cta(nch, local, pool=bool(seed & 1))
    progs = [rows(t), products(t), factors(t, 0), factors(t, 1)] + [norms(t, i) for i in range(NORMS)] + [worker(t, w) for w in range(t.workers)]
    speed = [rng.choice([0.02, 0.3, 1, 1]) for _ in progs] + [rng.choice([0.02, 0.3, 1])]  # the last: the tensor core
    wait = [None] * len(progs)
    alive = set(range(len(progs)))
    while alive or t.queue:
        able = [i for i in alive if wait[i] is None or t.bar[wait[i][0]].ready(wait[i][1])]
        if t.queue:
            able.append(len(progs))
        assert able, f"{nch} chunks, local {local}, seed {seed}: nothing can go on, waits {wait}"
        i = rng.choices(able, [speed[k] for k in able])[0]
        if i == len(progs):
            t.step_queue()
            continue
        wait[i] = None
        try:
            wait[i] = next(progs[i])
        except StopIteration:
            alive.discard(i)
            wait[i] = None


@pytest.mark.parametrize("local", [False, True])
@pytest.mark.parametrize("nch", [1, 2, 3, 4, 5, 9, 20])
def test_every_order_ends_and_overwrites_nothing(nch, local):
    for seed in range(150):
        run(nch, local, seed)
