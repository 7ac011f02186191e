"""The tensor core's order in the linear attention kernel (csrc/linattn_tc.cuh), on a model (CPU).

Only products of one shape on one accumulator run in the order of their issue.  Here the queue of the
model in test_linattn_protocol lets any others pass each other; what a product overwrites
must then be guarded by a wait.  The scores lie in P's columns, which the next chunk's QK
overwrites and, at d = 64, this chunk's U too: both wait until PV has read them."""
import random

import pytest

from tests.test_linattn_protocol import Bar, Model


class Unordered(list):
    """The tensor core's queue: a product waits for earlier ones on its accumulator, a commit for all
    earlier products, and nothing else is in order."""

    def __init__(self, rng):
        super().__init__()
        self.rng = rng

    @staticmethod
    def accumulator(op):
        return {"qk": "P", "pv": "O1", "xs": "O2"}.get(op[0]) or op[-1]

    def pop(self, _):
        may, busy = [], set()
        for i, op in enumerate(self):
            if op[0] == "commit":
                if not busy:
                    may.append(i)
            else:
                if self.accumulator(op) not in busy:
                    may.append(i)
                busy.add(self.accumulator(op))
        return super().pop(self.rng.choice(may))


class Issued(Model):
    """As the kernel issues: QK, and U where it lies in P, wait for PV's own barrier."""

    def __init__(self, rng, *a):
        super().__init__(rng, *a)
        self.queue = Unordered(rng)
        self.b["pv"] = Bar(1)

    def run_op(self, op):
        if op[0] == "up" and self.full and self.share_u and op[2] == 0:
            assert self.hold.get("P") == ("scores used", op[1]), "U overwrites scores that PV still reads"
        super().run_op(op)

    def pv_done(self, c):
        return c < 0 or self.b["pv"].passed(c)

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
                    self.issue(("pv", c), ("commit", "pv"))
                    pv = False
                if xs and not pv and self.b["s", c % 2].passed(c // 2):
                    self.issue(("xs", c), ("commit", "o"), ("commit", ("empty", (ty - 1) % self.slots)))
                    xs = False
                if (qk and not pv and self.pv_done(c)
                        and (not self.share_u or c < 0 or (not u and self.b["r", c % 2].passed(c // 2)))
                        and landed(3 * c + 3) and landed(3 * c + 4) and (c + 1 != self.ragged or self.b["z"].passed(0))):
                    self.issue(("qk", c + 1), ("commit", "qk"))
                    qk = False
                if (u and not pv and (not self.share_u or self.pv_done(c)) and self.b["y", step % 2].passed(step // 2)
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


class ByIssueAlone(Issued):
    """Without that wait: the order of issue is all that there is."""

    def pv_done(self, c):
        return True


def model(kind, d, full, seed):
    rng = random.Random(1000 * d + 10 * seed + full)
    n = rng.choice((0, 1, 2, 3, 5, 9))
    steps = [rng.choice((1, 2)) if d >= 64 else 1 for _ in range(n)]
    ragged = rng.choice((-1, 0, n - 1))
    return kind(rng, n, full, full and d == 64, d == 128, {128: 5, 64: 4, 32: 6}[d], steps, ragged)


@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("d", [128, 64, 32])
def test_products_that_pass_each_other(d, full):
    for seed in range(120):
        model(Issued, d, full, seed).run()


@pytest.mark.parametrize("d", [128, 64, 32])
def test_the_model_sees_products_out_of_order(d):
    """An issue that trusts the order of PV and what overwrites its scores is caught."""
    failed = 0
    for seed in range(40):
        try:
            model(ByIssueAlone, d, True, seed).run()
        except AssertionError:
            failed += 1
    assert failed > 0
