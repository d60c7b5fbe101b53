"""A model of the barriers of the feed-forward block's tensor-core kernels (csrc/ffn_tc.cu): the roles of
one CTA as generators that a random schedule steps, asynchronous copies and products as events that
take time, waits with a limit.

A wait tells a phase by its parity only, as in the kernel. run() raises Hang when no role can go on
and nothing is under way, Wrong when a role finds other data than its step needs although no wait
has run out, or when the kernel ends with a copy or a product in flight, or reports success without
its outputs. A copy or product that is `late` makes waits run out (by less than two limits: what is
in flight at the end is waited for twice as long as data, no longer).

Mistakes that can be planted: "meet" (the loader warps meet at a barrier without a limit, after a look
at the failure flag each on its own), "apart" (the lanes of a warp look at it each on its own), "silent"
(a wait for data that runs out says nothing), "go on" (a loader goes on after a staged tile that did not
come), "trust" (it goes by its barriers alone, which other roles move on after a failed wait), "count
skipped" (the weights waited for at the end include some that were not asked for after
a failed wait).
"""
import random

LIMIT = 10**6  # of a wait, in steps
PRODUCT, COPY = 12, 40  # steps that products and copies take


class Hang(Exception):
    pass


class Wrong(Exception):
    pass


class Bar:
    """An mbarrier: a phase is over when `count` arrivals and the expected copies are there."""

    def __init__(self, count=1):
        self.count, self.pending, self.open, self.phase = count, count, 0, 0

    def arrive(self):
        if self.pending == 0:
            raise Wrong("an arrival too many: the phase's copies are not there")
        self.pending -= 1
        self._turn()

    def expect(self, n=1):
        self.open += n

    def complete(self):
        self.open -= 1
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.open == 0:
            self.phase += 1
            self.pending = self.count

    def over(self, parity):  # the phase of this parity is over, as far as parity can tell
        return (self.phase & 1) != parity


class Plan:
    """What the host chooses: mode fwd | dx | dw, chunks, weight stages, row tiles, hidden operands,
    first-product accumulators, outputs, whether outputs have places of their own, whether rows come
    by staged copies."""

    def __init__(self, mode, nch, nt, nst, nx, nh, ngu, no, placed, staged):
        self.mode, self.nch, self.nt, self.nst, self.nx = mode, nch, nt, nst, nx
        self.nh, self.ngu, self.no, self.placed, self.staged = nh, ngu, no, placed, staged

    def __repr__(self):
        return f"Plan({', '.join(f'{k}={v!r}' for k, v in vars(self).items())})"


def random_plan(R):
    nt = R.randint(1, 9)
    staged = R.random() < 0.6
    if R.random() < 0.33:
        nx, nh = R.choice([(3, 2), (2, 2), (2, 1)])
        return Plan("dw", 1, nt, 1, nx, nh, R.randint(1, 3), 0, False, staged)
    nch = R.choice([1, 1, 2, 3, 4, 5, 8, 9, 16])
    nx, nh, placed = R.choice([(2, 2, True), (2, 2, False), (1, 2, True), (1, 2, False)])
    return Plan(R.choice(["fwd", "dx"]), nch, nt, R.randint(min(2, nch), nch), nx, nh,
                R.randint(2, 3), R.randint(1, 2), placed, staged)


class Cta:
    def __init__(self, plan, seed, late=None, mistakes=()):
        self.p, self.R, self.late, self.bad = plan, random.Random(seed), late, set(mistakes)
        self.now, self.events, self.started = 0, [], 0
        self.failed = self.status = False
        self.flight = {"copy": 0, "product": 0}
        self.deadlines = {}
        p = plan
        self.full = [Bar() for _ in range(p.nst)]
        self.empty = [Bar() for _ in range(p.nst)]
        self.gu_bars = max(p.ngu, 2)
        self.gu_full = [Bar() for _ in range(self.gu_bars)]
        self.gu_free = [Bar() for _ in range(p.ngu)]
        self.x_ready = [Bar(2) for _ in range(p.nx)]
        self.x_free = [Bar() for _ in range(p.nx)]
        self.h_ready, self.done, self.out_full, self.out_free = ([Bar(), Bar()] for _ in range(4))
        self.raw_full, self.all_done, self.read = Bar(), Bar(2), 0
        # what lies where
        self.W, self.X, self.raw = [None] * p.nst, [[None, None] for _ in range(p.nx)], None
        self.GU, self.H, self.A = [None] * p.ngu, [None] * p.nh, [None, None]
        self.outs, self.sums = [], []
        self.queue = {"first": [], "second": []}
        self.met = 0

    # -- time ---------------------------------------------------------------------------------
    def start(self, kind, effect, steps):
        """effect() after some steps (the `late`-th thing started: much later)"""
        self.flight[kind] += 1
        t = self.now + self.R.randint(1, steps)
        if self.late is not None and self.started == self.late[0]:
            t = self.now + self.late[1]
        self.started += 1

        def end():
            self.flight[kind] -= 1
            effect()
        self.events.append((t, self.started, end))

    def tick(self):
        self.now += 1
        due = sorted(e for e in self.events if e[0] <= self.now)
        for e in due:
            self.events.remove(e)
            e[2]()
        return due

    def need(self, ok, what):
        if not ok and not self.failed:
            raise Wrong(f"{what} in {self.p}")

    # -- waits --------------------------------------------------------------------------------
    def wait(self, bar, parity, silent=False, limit=LIMIT):
        t0, limit = None, limit + self.R.randint(0, 200)
        while not bar.over(parity & 1):
            if self.failed and not silent:
                return False
            if t0 is None:
                t0 = self.now
                yield None  # (what came before this wait was a step)
                continue
            if self.now - t0 > limit:
                if not silent:
                    self.failed = True
                    self.status = True
                return False
            yield t0 + limit + 1
        yield None
        return True

    def drain(self, bar, parity):  # before the end: what is in flight
        yield from self.wait(bar, parity, silent=True, limit=2 * LIMIT)

    def stop(self):
        """A warp's common look at the failure flag."""
        first = self.failed
        for _ in range(self.R.randint(1, 4)):
            yield None
        second = self.failed
        if "apart" in self.bad and first != second:
            raise Hang("lanes of one warp went separate ways")
        return first or second

    # -- roles --------------------------------------------------------------------------------
    def product_warp(self):
        p, total, ring = self.p, self.p.nt * self.p.nch, self.p.nch > self.p.nst
        j = c1 = x1 = px = pw = 0
        gu, s1, pg, pe = 0, 0, 1, 1
        sj = loads = 0

        def load():
            nonlocal j, sj, pe, loads
            if not (yield from self.stop()):
                loads += 1
                c, s = j % p.nch, sj
                self.full[s].expect()
                self.full[s].arrive()
                self.W[s] = None

                def there():
                    self.W[s] = c
                    self.full[s].complete()
                self.start("copy", there, COPY)
            j += 1
            sj += 1
            if sj == p.nst:
                sj, pe = 0, pe ^ 1
            yield None
        uses = total if ring else p.nch
        while j < p.nst:
            yield from load()
        for i in range(total):
            if ring and j < uses:
                must = j <= i
                if must:
                    yield from self.wait(self.empty[sj], pe)
                if must or self.empty[sj].over(pe):
                    yield from load()
            if ring or i < p.nch:
                yield from self.wait(self.full[s1], pw)
            if c1 == 0:
                yield from self.wait(self.x_ready[x1], px)
            yield from self.wait(self.gu_free[gu], pg)
            self.issue("first", (i, gu, x1, s1, c1, i // p.nch))
            yield None
            gu += 1
            if gu == p.ngu:
                gu, pg = 0, pg ^ 1
            s1 += 1
            if s1 == p.nst:
                s1, pw = 0, pw ^ 1
            c1 += 1
            if c1 == p.nch:
                c1, x1 = 0, x1 + 1
                if x1 == p.nx:
                    x1, px = 0, px ^ 1
        if "count skipped" in self.bad:
            loads = j
        for k in range(max(0, loads - p.nst), loads):
            yield from self.drain(self.full[k % p.nst], k // p.nst)
        self.issue("first", None)

    def second_warp(self):
        p, total = self.p, self.p.nt * self.p.nch
        hb = x2 = s2 = o2 = 0
        po = 1
        for i in range(total):
            c = i % p.nch
            yield from self.wait(self.h_ready[i & 1], i >> 1)
            if p.mode != "dw" and c == 0:
                yield from self.wait(self.out_free[o2], po)
            self.issue("second", (i, hb, x2, s2, o2, c, i // p.nch))
            yield None
            hb, s2 = (hb + 1) % p.nh, (s2 + 1) % p.nst
            if c == p.nch - 1:
                x2 = (x2 + 1) % p.nx
                o2 += 1
                if o2 == p.no:
                    o2, po = 0, po ^ 1

    def issue(self, kind, op):
        """Products of one warp run in order, each some steps after the one before."""
        q = self.queue[kind]
        q.append(op)
        if len(q) == 1:
            self.begin(kind)

    def begin(self, kind):
        op, p = self.queue[kind][0], self.p
        if op is None:
            self.queue[kind].pop(0)
            self.all_done.arrive()
            return
        if kind == "first":
            i, gu, x, s, c, n = op
            self.need(self.X[x] == [n, n], f"first product {op}: rows {self.X[x]}")
            self.need(self.W[s] == c, f"first product {op}: weights {self.W[s]}")
        else:
            i, hb, x, s, o, c, n = op
            self.need(self.H[hb] == i, f"second product {op}: operand {self.H[hb]}")
            if p.mode == "dw":
                self.need(self.X[x] == [n, n], f"second product {op}: rows {self.X[x]}")
                self.sums.append((n, not self.failed and self.H[hb] == i))
            else:
                self.need(self.W[s] == c, f"second product {op}: weights {self.W[s]}")
                self.need(self.A[o] == (None if c == 0 else (n, c)), f"{op}: output {self.A[o]}")

        def end():
            if kind == "first":
                self.need(self.X[x] == [n, n], f"first product {op}: rows taken away")
                self.GU[gu] = i
                self.gu_full[i % self.gu_bars].arrive()
                if p.mode != "dw" and c == p.nch - 1:
                    self.x_free[x].arrive()
            else:
                self.need(self.H[hb] == i, f"second product {op}: operand taken away")
                if p.mode == "dw":
                    self.need(self.X[x] == [n, n], f"second product {op}: rows taken away")
                    self.x_free[x].arrive()
                else:
                    self.A[o] = (n, c + 1)
                    if c == p.nch - 1:
                        self.out_full[o].arrive()
                self.done[i & 1].arrive()
                if p.nch > p.nst:
                    self.empty[s].arrive()
                if i == p.nt * p.nch - 1:
                    self.all_done.arrive()
            self.queue[kind].pop(0)
            if self.queue[kind]:
                self.begin(kind)
        self.start("product", end, PRODUCT)

    def loader(self, w):
        p = self.p
        xb, pf, taken, staged_tile = 0, 1, 0, 0
        half = w  # each warp lays out half the rows

        def fetch(n):
            self.raw_full.expect()
            self.raw_full.arrive()
            self.raw = None

            def there():
                self.raw = n
                self.raw_full.complete()
            self.start("copy", there, COPY)
        if p.staged and w == 0:
            fetch(0)
        for n in range(p.nt):
            over = yield from self.wait(self.x_free[xb], pf)
            if "trust" in self.bad:
                if not over:
                    break
            elif (yield from self.stop()):
                break
            came = True
            if not p.staged:
                if w == 0:
                    b = xb
                    self.X[b] = ["filling"] * 2
                    self.x_ready[b].expect()

                    def there(b=b, n=n):
                        self.X[b] = [n, n]
                        self.x_ready[b].complete()
                    self.start("copy", there, COPY)
                yield None
            else:
                self.X[xb][half] = "filling"
                came = yield from self.wait(self.raw_full, n, silent="silent" in self.bad)
                came |= bool({"silent", "go on"} & self.bad)
                staged_tile = n
                for _ in range(2):
                    self.need(self.raw == n, f"staged tile {n}: {self.raw}")
                    right = self.raw == n
                    yield None
                self.X[xb][half] = n if right and self.raw == n else "torn"
            self.x_ready[xb].arrive()
            if p.staged and n + 1 < p.nt:
                yield None
                if "meet" in self.bad:
                    self.met += 1
                    want = (self.met + 1) // 2 * 2
                    while self.met < want:
                        yield "forever"
                    if w == 0:
                        fetch(n + 1)
                        staged_tile = n + 1
                else:
                    self.read += 1
                    if self.read == 2 * n + 2 and came:
                        fetch(n + 1)
                        staged_tile = n + 1
            xb += 1
            if xb == p.nx:
                xb, pf = 0, pf ^ 1
            taken += 1
            if not came:
                break
        for n in range(max(0, taken - p.nx), taken):
            yield from self.drain(self.x_ready[n % p.nx], n // p.nx)
        if p.staged:
            yield from self.drain(self.raw_full, staged_tile)

    def group(self, g):
        p, total = self.p, self.p.nt * self.p.nch

        def output(n, i):
            if p.placed:
                if i == total and total >= 2:
                    e = (total - 1 - g) // 2 * 2 + g
                    yield from self.wait(self.done[e & 1], e >> 1)
                yield from self.wait(self.out_full[n % p.no], n // p.no)
            else:
                yield from self.wait(self.done[i & 1], i >> 1)
            self.need(self.A[n % p.no] == (n, p.nch), f"output {n}: {self.A}")
            right = self.A[n % p.no] == (n, p.nch)
            if not p.placed:
                self.H[i % p.nh] = ("out", n)
            yield None
            self.A[n % p.no] = None
            self.out_free[n % p.no].arrive()
            yield None
            if not p.placed:
                self.need(self.H[i % p.nh] == ("out", n), f"output {n}: its place {self.H}")
            self.outs.append((n, right))
        for i in range(g, total, 2):
            n, c = i // p.nch, i % p.nch
            yield from self.wait(self.gu_full[i % self.gu_bars], i // self.gu_bars)
            self.need(self.GU[i % p.ngu] == i, f"item {i}: accumulator {self.GU}")
            if i >= p.nh:
                yield from self.wait(self.done[(i - p.nh) & 1], (i - p.nh) >> 1)
            self.H[i % p.nh] = "filling"
            yield None
            self.need(self.GU[i % p.ngu] == i, f"item {i}: accumulator taken away")
            right = self.GU[i % p.ngu] == i
            self.gu_free[i % p.ngu].arrive()
            yield None
            self.H[i % p.nh] = i if right else "wrong"
            self.h_ready[i & 1].arrive()
            yield None
            if p.mode != "dw":
                if not p.placed:
                    if c == p.nch - 1:
                        yield from output(n, i)
                elif c < 2 and n > 0 and (p.nch == 1 or ((n - 1) & 1) == g):
                    yield from output(n - 1, i)
        if p.mode != "dw" and p.placed and g == (p.nt & 1 if p.nch == 1 else (p.nt - 1) & 1):
            yield from output(p.nt - 1, total)
        if p.mode == "dw" and g == 0:
            yield from self.wait(self.all_done, 0, silent="silent" in self.bad)
            self.need(len(self.sums) == p.nt and self.flight["product"] == 0, "sums read early")
            self.outs = [(n, ok and self.flight["product"] == 0) for n, ok in self.sums]

    def run(self):
        self.steps({"products": self.product_warp(), "second": self.second_warp(),
                    "loader 0": self.loader(0), "loader 1": self.loader(1),
                    "group 0": self.group(0), "group 1": self.group(1)})
        self.steps({"end": self.drain(self.all_done, 0)})  # before TMEM is given back
        if self.flight["copy"] or self.flight["product"]:
            raise Wrong(f"the CTA ended with {self.flight} in flight: {self.p}")
        if not self.status and sorted(self.outs) != [(n, True) for n in range(self.p.nt)]:
            raise Wrong(f"success without its results: {self.outs} of {self.p}")
        return self.status

    def steps(self, roles):
        weight = {k: self.R.choice([1, 3, 10]) for k in roles}
        blocked = {}  # role -> when its wait runs out
        while roles:
            names = list(roles)
            k = self.R.choices(names, [weight[n] for n in names])[0]
            if self.tick():
                blocked.clear()
            try:
                r = next(roles[k])
            except StopIteration:
                del roles[k]
                blocked.pop(k, None)
                continue
            if r is None:
                blocked.clear()
                continue
            blocked[k] = r
            if len(blocked) == len(roles):  # nothing but time can help
                limits = [t for t in blocked.values() if t != "forever"]
                times = limits + [e[0] for e in self.events]
                if not times:
                    raise Hang(f"{sorted(roles)} in {self.p}")
                self.now = max(self.now, min(times) - 1)
                blocked.clear()
