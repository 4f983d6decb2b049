"""The barrier protocol of the packed attention kernel, replayed on the CPU: its roles (loads, S issuer, P.V issuer,
the two softmax groups) as generators that wait on mbarriers by parity and arrive on them in the kernel's order, under
random schedules and lists of items.  It checks that no schedule deadlocks, and that every buffer holds what its
reader expects: S and P buffers of the right block, O complete before it is rescaled or stored, the row maxima and
sums of the right block and item.  (A wait by parity passes wrongly when it runs two phases ahead: the replay sees
that too.)"""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):  # mbarrier.try_wait.parity
        return (self.phase & 1) != parity


def replay(items, k_stages, v_stages, rng, raises):
    bars = {}

    def bar(*names, count=1):
        for n in names:
            bars[n] = Bar(count)

    for i in range(2):
        bar(("QF", i), ("QE", i), ("SF", i), ("SE", i), ("PF", i), ("PE", i), ("MX", i))
    for i in range(k_stages):
        bar(("KF", i), ("KE", i))
    for i in range(v_stages):
        bar(("VF", i), ("VE", i))
    bar("SUM", "OE", count=2)
    bar("OF")
    S, P, O, sums, maxima = [None] * 2, [None] * 2, [None, 2], {}, {}
    done = [-1]  # the last block whose P.V product is complete
    blocks = [(n, j, b) for n, b in enumerate(items) for j in range(b)]

    def loads():
        gk = 0

        def next_k():
            nonlocal gk
            if gk == len(blocks):
                return
            n, j, _ = blocks[gk]
            if j == 0:
                yield ("QE", n & 1), ((n >> 1) & 1) ^ 1
                bars[("QF", n & 1)].arrive()
            yield ("KE", gk % k_stages), ((gk // k_stages) & 1) ^ 1
            bars[("KF", gk % k_stages)].arrive()
            gk += 1

        for _ in range(2):
            yield from next_k()
        for gv in range(len(blocks)):
            yield from next_k()
            yield ("VE", gv % v_stages), ((gv // v_stages) & 1) ^ 1
            bars[("VF", gv % v_stages)].arrive()

    def s_issuer():
        for g, (n, j, b) in enumerate(blocks):
            if j == 0:
                yield ("QF", n & 1), (n >> 1) & 1
            yield ("KF", g % k_stages), (g // k_stages) & 1
            yield ("SE", g & 1), ((g >> 1) & 1) ^ 1
            assert S[g & 1] is None
            S[g & 1] = g
            bars[("SF", g & 1)].arrive()
            bars[("KE", g % k_stages)].arrive()
            if j == b - 1:
                bars[("QE", n & 1)].arrive()

    def pv_issuer():
        for g, (n, j, b) in enumerate(blocks):
            yield ("VF", g % v_stages), (g // v_stages) & 1
            if j == 0:
                yield "OE", (n & 1) ^ 1
            yield ("PF", g & 1), (g >> 1) & 1
            assert P[g & 1] == g
            if j == 0:
                assert O[1] == 2  # both groups have stored the item before
                O[:] = [n, 0]
            P[g & 1], done[0] = None, g
            bars[("PE", g & 1)].arrive()
            bars[("VE", g % v_stages)].arrive()
            if j == b - 1:
                bars["OF"].arrive()

    def softmax(x):
        g = n = 0
        pending = False

        def epilogue():
            nonlocal pending
            pending, k = False, n - 1
            yield "SUM", k & 1
            assert sums[(k & 1, 0)] == sums[(k & 1, 1)] == k
            yield "OF", k & 1
            assert O[0] == k
            O[1] += 1
            bars["OE"].arrive()

        for b in items:
            for j in range(b):
                if (g & 1) == x:
                    use = (g >> 1) & 1
                    yield ("SF", x), use
                    assert S[x] == g
                    if g > 0:
                        yield ("MX", (g - 1) & 1), ((g - 1) >> 1) & 1
                        assert maxima[(g - 1) & 1] == g - 1
                    maxima[g & 1] = g
                    bars[("MX", g & 1)].arrive()
                    if j > 0 and rng.random() < raises:
                        if pending:
                            yield from epilogue()
                        yield ("PE", x), use ^ 1
                        yield ("PE", (g - 1) & 1), ((g - 1) >> 1) & 1
                        assert done[0] == g - 1
                    S[x] = None
                    bars[("SE", x)].arrive()
                    yield None
                    yield ("PE", x), use ^ 1
                    assert P[x] is None
                    P[x] = g
                    bars[("PF", x)].arrive()
                    if pending:
                        yield from epilogue()
                g += 1
            if pending:
                yield from epilogue()
            sums[(n & 1, x)] = n
            bars["SUM"].arrive()
            pending, n = True, n + 1
        if pending:
            yield from epilogue()

    roles = [loads(), s_issuer(), pv_issuer(), softmax(0), softmax(1)]
    waits = [next(r, "end") for r in roles]
    while any(w != "end" for w in waits):
        ready = [i for i, w in enumerate(waits) if w != "end" and (w is None or bars[w[0]].done(w[1]))]
        assert ready, ("deadlock", waits, items)
        i = rng.choice(ready)
        waits[i] = next(roles[i], "end")
    assert O == [len(items) - 1, 2] or not items


@pytest.mark.parametrize("stages", [(2, 2), (4, 4)])  # head_dim 96 and 128, 64
@pytest.mark.parametrize("raises", [0.0, 0.3, 1.0])
def test_every_schedule_ends(stages, raises):
    rng = random.Random(f"{stages} {raises}")
    for _ in range(300):
        items = [rng.choice((1, 1, 2, 3, rng.randint(1, 9))) for _ in range(rng.randint(0, 9))]
        replay(items, *stages, rng, raises)
