"""The packed attention kernel's way out of a wait that runs out, replayed on the CPU: its roles as in
test_packed_protocol.py, with one arrival lost at random.  Some wait then never ends by itself; its limit sets the
abort flag.  Every role has to leave with the item it is in, however long its list of items."""
import random

import pytest
from test_packed_protocol import Bar

BLOCK_WAITS = 5  # of a softmax group in a block at most, each returning at its first look after the abort


class Replay:
    def __init__(self, items, k_stages, v_stages, rng, raises, lost):
        self.items, self.rng, self.raises, self.lost = items, rng, raises, lost
        self.ks, self.vs, self.gone, self.arrivals = k_stages, v_stages, False, 0
        self.blocks = [(n, j, b) for n, b in enumerate(items) for j in range(b)]
        self.bars = {}
        for i in range(2):
            for n in ("QF", "QE", "SF", "SE", "PF", "PE", "MX"):
                self.bars[n, i] = Bar(1)
        for i in range(k_stages):
            self.bars["KF", i], self.bars["KE", i] = Bar(1), Bar(1)
        for i in range(v_stages):
            self.bars["VF", i], self.bars["VE", i] = Bar(1), Bar(1)
        self.bars["SUM"], self.bars["OE"], self.bars["OF"] = Bar(2), Bar(2), Bar(1)

    def arrive(self, name):
        self.arrivals += 1
        if self.arrivals != self.lost:
            self.bars[name].arrive()

    # a wait yields (barrier, parity) and receives whether the phase completed
    def loads(self):
        gk = 0

        def next_k():
            nonlocal gk
            if gk == len(self.blocks):
                return True
            n, j, _ = self.blocks[gk]
            if j == 0:
                if not (yield ("QE", n & 1), ((n >> 1) & 1) ^ 1):
                    return False
                self.arrive(("QF", n & 1))
            if not (yield ("KE", gk % self.ks), ((gk // self.ks) & 1) ^ 1):
                return False
            self.arrive(("KF", gk % self.ks))
            gk += 1
            return True

        for _ in range(2):
            if not (yield from next_k()):
                return
        for gv in range(len(self.blocks)):
            if not (yield from next_k()) or not (yield ("VE", gv % self.vs), ((gv // self.vs) & 1) ^ 1):
                return
            self.arrive(("VF", gv % self.vs))

    def s_issuer(self):
        for g, (n, j, b) in enumerate(self.blocks):
            if j == 0 and not (yield ("QF", n & 1), (n >> 1) & 1):
                return
            if not (yield ("KF", g % self.ks), (g // self.ks) & 1) or not (yield ("SE", g & 1), ((g >> 1) & 1) ^ 1):
                return
            self.arrive(("SF", g & 1))
            self.arrive(("KE", g % self.ks))
            if j == b - 1:
                self.arrive(("QE", n & 1))

    def pv_issuer(self):
        for g, (n, j, b) in enumerate(self.blocks):
            if not (yield ("VF", g % self.vs), (g // self.vs) & 1):
                return
            if j == 0 and not (yield "OE", (n & 1) ^ 1):
                return
            if not (yield ("PF", g & 1), (g >> 1) & 1):
                return
            self.arrive(("PE", g & 1))
            self.arrive(("VE", g % self.vs))
            if j == b - 1:
                self.arrive("OF")

    def softmax(self, x):
        """Waits are not looked at one by one: the abort flag is, before a store or a rescaling and at an item's end."""
        g = n = 0
        pending = False

        def epilogue():
            nonlocal pending
            pending, k = False, n - 1
            yield "SUM", k & 1
            yield "OF", k & 1
            if self.gone:
                return
            yield None  # the loads and stores of a tile
            self.arrive("OE")

        for b in self.items:
            for j in range(b):
                if (g & 1) == x:
                    use = (g >> 1) & 1
                    yield ("SF", x), use
                    if g > 0:
                        yield ("MX", (g - 1) & 1), ((g - 1) >> 1) & 1
                    self.arrive(("MX", g & 1))
                    if j > 0 and self.rng.random() < self.raises:
                        if pending:
                            yield from epilogue()
                        yield ("PE", x), use ^ 1
                        yield ("PE", (g - 1) & 1), ((g - 1) >> 1) & 1
                        if self.gone:
                            break
                    self.arrive(("SE", x))
                    yield ("PE", x), use ^ 1
                    self.arrive(("PF", x))
                    if pending:
                        yield from epilogue()
                g += 1
            if self.gone:
                break
            if pending:
                yield from epilogue()
            self.arrive("SUM")
            pending, n = True, n + 1
        if pending:
            yield from epilogue()

    def run(self):
        roles = [self.loads(), self.s_issuer(), self.pv_issuer(), self.softmax(0), self.softmax(1)]
        waits = [next(r, "end") for r in roles]
        after = [0] * 5

        def step(i, ok):
            try:
                waits[i] = roles[i].send(ok)
            except StopIteration:
                waits[i] = "end"
            if self.gone and waits[i] not in ("end", None):
                after[i] += 1

        while any(w != "end" for w in waits):
            open_ = [i for i, w in enumerate(waits) if w != "end"]
            ready = [i for i in open_ if waits[i] is None or self.bars[waits[i][0]].done(waits[i][1])]
            if self.gone:  # a wait that is not ready gives up at its next look
                i = self.rng.choice(open_)
                step(i, i in ready)
            elif ready:
                step(self.rng.choice(ready), True)
            else:  # nothing moves: the limit of one of the waits
                i = self.rng.choice(open_)
                self.gone = True
                step(i, False)
        # the loader and the issuers leave at their first wait that is not ready, at most a ring's stages ahead (three
        # waits a block, K and V each); the groups leave with the item they are in and its epilogue
        assert all(a <= 3 * (self.ks + self.vs) for a in after[:3]), after
        assert all(a <= BLOCK_WAITS * max(self.items, default=0) + 4 for a in after[3:]), after
        return self.gone


@pytest.mark.parametrize("stages", [(2, 2), (4, 4)])
@pytest.mark.parametrize("raises", [0.0, 0.3, 1.0])
def test_every_role_leaves_after_a_wait_that_runs_out(stages, raises):
    rng = random.Random(f"abort {stages} {raises}")
    stuck = 0
    for _ in range(400):
        items = [rng.choice((1, 1, 2, 3, rng.randint(1, 9))) for _ in range(rng.randint(1, 9))]
        stuck += Replay(items, *stages, rng, raises, rng.randint(1, 14 * sum(items))).run()
    assert stuck > 200  # most lost arrivals are waited for


def test_nothing_is_lost_without_a_lost_arrival():
    rng = random.Random(3)
    for _ in range(100):
        items = [rng.randint(1, 5) for _ in range(rng.randint(0, 9))]
        assert not Replay(items, 2, 2, rng, 0.5, -1).run()
