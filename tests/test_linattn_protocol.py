"""A model of the tensor-core linear attention kernel's waits (csrc/linattn_tc.cuh) under random
schedules (CPU).

The kernel's roles wait on mbarriers by parity alone: a waiter that falls two phases behind
would take the wrong phase for its own, and a buffer that is reused too early would go
unnoticed.  Here each role is a generator that makes the kernel's waits, arrivals, tensor-core
products (run in order by a queue) and copies (finished in any order); a scheduler steps them at
random.  Every buffer knows what it holds, so each read checks that it gets the chunk that it
means and each write that nobody still reads what it replaces."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, "an arrival too many"
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, phase):
        """What a parity wait sees, and whether it is the truth."""
        seen = self.phase % 2 != phase % 2
        if seen:
            assert self.phase > phase, "a wait took another phase for its own"
        return seen


class Model:
    def __init__(self, rng, chunks, full, share_u, out_s, slots, steps, ragged):
        self.rng, self.n, self.full, self.share_u, self.out_s, self.slots = rng, chunks, full, share_u, out_s, slots
        self.steps, self.ragged = steps, ragged                 # steps a chunk; the ragged chunk or -1
        b = self.b = {k: Bar(1) for k in ("qk", "o", "sent", "end")}
        self.wa, self.wb = 2, 2
        b["p"], b["z"], b["out"] = Bar(self.wa), Bar(self.wa), Bar(self.wb)
        for i in (0, 1):
            b["t", i], b["u", i], b["y", i] = Bar(1), Bar(1), Bar(self.wa)
            b["s", i], b["r", i] = Bar(self.wb), Bar(self.wb)
        for s in range(slots):
            b["full", s], b["empty", s] = Bar(1), Bar(1)
        self.hold = {}                                          # buffer -> what it holds
        self.queue, self.copies, self.stores = [], [], []
        self.split = {}                                         # (chunk, step) -> A's warps that wrote it
        self.got = {"O": [], "U": [], "S": []}

    def put(self, where, what):
        self.hold[where] = what

    def want(self, where, what):
        assert self.hold.get(where) == what, f"{where} holds {self.hold.get(where)}, not {what}"

    # -- tensor core: in order --
    def issue(self, *ops):
        self.queue.extend(ops)

    def run_op(self, op):
        kind = op[0]
        if kind == "commit":
            self.b[op[1]].arrive()
        elif kind == "qk":
            c = op[1]
            self.want(("slot", 3 * c % self.slots), ("x", c))
            self.want(("slot", (3 * c + 1) % self.slots), ("y", c))
            assert self.hold.get("P") in (None, ("scores used", c - 1)), "P is overwritten"
            if self.share_u:
                assert self.hold.get("U0") in (None, ("read", c - 1)), "P over a U that is not read"
            self.put("P", ("P", c))
        elif kind == "pv":
            c = op[1]
            self.want("P", ("scores", c))
            self.want(("slot", (3 * c + 2) % self.slots), ("z", c))
            assert self.hold.get("O1") in (None, ("read", c - 1)), "O1 is overwritten"
            self.put("O1", ("O", c))
            self.put("P", ("scores used", c))
        elif kind == "xs":
            c = op[1]
            self.want(("slot", 3 * c % self.slots), ("x", c))
            self.want("S", ("state", c))
            assert self.hold.get("O2") in (None, ("read", c - 1)), "O2 is overwritten"
            self.put("O2", ("O", c))
            self.put("S", ("used", c))
        else:
            c, k, step, terms, u = op[1:]
            self.want(("terms", terms), ("terms", step))
            tz = 3 * c + 2 if self.full else 2 * c + 1
            self.want(("slot", tz % self.slots), ("z", c))
            if k == 0:
                old = self.hold.get(u)
                assert old is None or old[0] == "read", "U is overwritten"
            else:
                self.want(u, ("sum", c, k - 1))
            self.put(u, ("sum", c, k))
            self.put(("terms", terms), ("used", step))

    # -- roles --
    def wait(self, bar, phase):
        while not self.b[bar].passed(phase):
            yield
        yield

    def copier(self):
        per = 3 if self.full else 2
        for tile in range(self.n * per):
            s = tile % self.slots
            if tile >= self.slots:
                yield from self.wait(("empty", s), tile // self.slots - 1)
            name = ("xyz" if self.full else "yz")[tile % per]
            self.copies.append((s, (name, tile // per)))
            yield

    def mma(self):
        per, step = (3 if self.full else 2), 0

        def landed(tile):
            return self.b["full", tile % self.slots].passed(tile // self.slots)

        for c in range(-1 if self.full else 0, self.n):
            ty = per * c + per - 2
            pv = xs = self.full and c >= 0
            qk, u, k = self.full and c + 1 < self.n, c >= 0, 0
            last = c - 1 if self.full else c - 2
            while pv or xs or qk or u:
                yield
                if pv and landed(ty + 1) and self.b["p"].passed(c) and (c == 0 or self.b["out"].passed(c - 1)):
                    self.issue(("pv", c))
                    pv = False
                if xs and not pv and self.b["s", c % 2].passed(c // 2):
                    self.issue(("xs", c), ("commit", "o"), ("commit", ("empty", (ty - 1) % self.slots)))
                    xs = False
                if (qk and not pv and (not self.share_u or c < 0 or (not u and self.b["r", c % 2].passed(c // 2)))
                        and landed(3 * c + 3) and landed(3 * c + 4) and (c + 1 != self.ragged or self.b["z"].passed(0))):
                    self.issue(("qk", c + 1), ("commit", "qk"))
                    qk = False
                if (u and not pv and self.b["y", step % 2].passed(step // 2)
                        and (last < 0 or k > 0 or self.b["r", last % 2].passed(last // 2))
                        and (self.full or (landed(ty + 1) and (c != self.ragged or self.b["z"].passed(0))))):
                    terms, where = (0 if self.full else step % 2), "U0" if self.full or c % 2 == 0 else "U1"
                    self.issue(("up", c, k, step, terms, where), ("commit", ("t", step % 2)))
                    step, k = step + 1, k + 1
                    if k == self.steps[c]:
                        self.issue(("commit", ("u", c % 2)), ("commit", ("empty", ty % self.slots)),
                                   ("commit", ("empty", (ty + 1) % self.slots)))
                        u = False
        self.issue(("commit", "end"))
        yield from self.wait("end", 0)

    def a_warp(self, w):
        per, step = (3 if self.full else 2), 0
        for c in range(self.n):
            ty = per * c + per - 2
            yield from self.wait(("full", ty % self.slots), ty // self.slots)
            if c == self.ragged:
                yield from self.wait(("full", (ty + 1) % self.slots), (ty + 1) // self.slots)
                self.b["z"].arrive()
                yield from self.wait("z", 0)
            if self.full:
                yield from self.wait("qk", c)
                self.want("P", ("P", c)) if w == 0 else None
                self.split.setdefault(("P", c), set()).add(w)
                if len(self.split["P", c]) == self.wa:
                    self.put("P", ("scores", c))
                self.b["p"].arrive()
                yield
            for k in range(self.steps[c]):
                back = 1 if self.full else 2
                if step >= back:
                    yield from self.wait(("t", (step - back) % 2), (step - back) // 2)
                self.want(("slot", ty % self.slots), ("y", c))
                terms = 0 if self.full else step % 2
                old = self.hold.get(("terms", terms))
                assert old is None or old == ("used", step - back) or old == ("part", step), "terms are overwritten"
                mine = self.split.setdefault(step, set())
                mine.add(w)
                self.put(("terms", terms), ("terms" if len(mine) == self.wa else "part", step))
                yield
                self.b["y", step % 2].arrive()
                step += 1

    def outputs(self, w, c):
        yield from self.wait("o", c)
        where = "S" if self.out_s else "out"
        old = self.hold.get(where)
        assert old in (None, ("used", c), ("sent", c - 1), ("part out", c)), f"{where} is overwritten: {old}"
        if w == 0:
            self.want("O1", ("O", c))
            self.want("O2", ("O", c))
        done = self.split.setdefault(("O", c), set())
        done.add(w)
        self.put(where, ("out" if len(done) == self.wb else "part out", c))
        if len(done) == self.wb:
            self.put("O1", ("read", c))
            self.put("O2", ("read", c))
        yield
        self.b["out"].arrive()

    def b_warp(self, w):
        for c in range(-1, self.n):
            if c >= 0:
                if self.full:
                    yield from self.outputs(w, c)
                if self.full and w == 0:
                    yield from self.wait("out", c)
                    self.want("S" if self.out_s else "out", ("out", c))
                    self.stores.append(c)
                    yield
                yield from self.wait(("u", c % 2), c // 2)
                u = "U0" if self.full or c % 2 == 0 else "U1"
                read = self.split.setdefault(("U", c), set())
                read.add(w)
                self.want(u, ("sum", c, self.steps[c] - 1))
                if len(read) == self.wb:
                    self.put(u, ("read", c))
                    self.got["U"].append(c)
                yield
                self.b["r", c % 2].arrive()
                if self.full:
                    if w == 0:
                        while c in self.stores:
                            yield
                        self.b["sent"].arrive()
                        yield
                    if self.out_s:
                        yield from self.wait("sent", c)
            if self.full:
                old = self.hold.get("S")
                ok = (None, ("part state", c + 1), ("sent", c)) if self.out_s else (None, ("part state", c + 1), ("used", c))
                assert old in ok, f"S is overwritten: {old}"
                wrote = self.split.setdefault(("S", c + 1), set())
                wrote.add(w)
                self.put("S", ("state" if len(wrote) == self.wb else "part state", c + 1))
                yield
                self.b["s", (c + 1) % 2].arrive()

    def run(self):
        roles = [self.copier(), self.mma()] + [self.a_warp(w) for w in range(self.wa)]
        roles += [self.b_warp(w) for w in range(self.wb)]
        speed = [self.rng.choice((1, 1, 3, 20)) for _ in range(len(roles) + 3)]
        idle = 0
        while roles or self.queue or self.copies or self.stores:
            kinds = list(range(len(roles))) + [-1] * bool(self.queue) + [-2] * bool(self.copies) + [-3] * bool(self.stores)
            at = self.rng.choices(kinds, [speed[k] for k in kinds])[0]
            before = {k: (v.phase, v.left) for k, v in self.b.items()}, len(self.queue), len(self.copies), len(self.stores), len(roles)
            if at == -1:
                self.run_op(self.queue.pop(0))
            elif at == -2:
                s, what = self.copies.pop(self.rng.randrange(len(self.copies)))
                self.put(("slot", s), what)
                self.b["full", s].arrive()
            elif at == -3:
                c = self.stores.pop(0)
                where = "S" if self.out_s else "out"
                self.want(where, ("out", c))
                self.put(where, ("sent", c))
                self.got["O"].append(c)
            else:
                try:
                    next(roles[at])
                except StopIteration:
                    del roles[at], speed[at]
            after = {k: (v.phase, v.left) for k, v in self.b.items()}, len(self.queue), len(self.copies), len(self.stores), len(roles)
            idle = 0 if after != before else idle + 1
            assert idle < 20000, "no role gets on"
        assert self.got["U"] == list(range(self.n)) and (not self.full or self.got["O"] == list(range(self.n)))


@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("d", [128, 64, 32])
def test_random_schedules(d, full):
    for seed in range(120):
        rng = random.Random(1000 * d + 10 * seed + full)
        n = rng.choice((0, 1, 2, 3, 5, 9))
        steps = [rng.choice((1, 2)) if d >= 64 else 1 for _ in range(n)]
        ragged = rng.choice((-1, 0, n - 1))
        Model(rng, n, full, full and d == 64, d == 128, {128: 5, 64: 4, 32: 6}[d], steps, ragged).run()


def test_the_model_sees_a_wait_that_is_two_phases_behind():
    """One barrier for all steps of the states' own launch: A may be two steps ahead of the
    issuing warp, whose parity wait then mistakes the phase or never ends."""
    class One(Model):
        def __init__(self, *a):
            super().__init__(*a)
            self.b["y", 0] = self.b["y", 1] = Bar(self.wa)

    failed = 0
    for seed in range(40):
        m = One(random.Random(seed), 9, False, False, True, 5, [1] * 9, -1)
        y = m.b["y", 0]
        # both parities' waits go to the one barrier, with the step's own number
        ask = y.passed
        m.b["y", 0] = type("Even", (), {"passed": lambda s, p: ask(2 * p), "arrive": lambda s: y.arrive(), "phase": 0, "left": 0})()
        m.b["y", 1] = type("Odd", (), {"passed": lambda s, p: ask(2 * p + 1), "arrive": lambda s: y.arrive(), "phase": 0, "left": 0})()
        try:
            m.run()
        except AssertionError:
            failed += 1
    assert failed > 0
