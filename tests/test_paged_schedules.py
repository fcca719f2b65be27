"""The barrier protocols of the two paged attention kernels, run through random schedules on the CPU.

A role of a kernel (a warp, or one of several alike) is a generator: it yields the barrier phase it
waits for and touches what the roles share in between. Copies land and products complete in order
but at any time after they were issued. Roles run at random speeds, some far slower than others.
A schedule fails if
- a role waits for a phase that is two or more behind the barrier: the kernels tell phases apart by
  parity, so that wait would not end;
- nobody can go on;
- a product, a softmax warp or a storing warp finds anything but what it is for (a tile, queries,
  S, P, O, sums, the list of loaded pages).

Each wait that keeps a role from running ahead is also left out once, in the model: the schedules
must find that, or they would not find a real one either. (Not so the waits for s_free and o_free
in the kernel for few rows, which others imply: chunk 7 of a block is loaded once PV of the block
two back is done, so after its softmax; PV of a unit's first block waits for the P of warps that
have stored the unit before.) Four warps that share a barrier's phase are two here."""
import random

import pytest


class Bar:
    def __init__(self, count=1):
        self.count, self.arrived, self.phase = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived = 0
            self.phase += 1


class Machine:
    """Roles, copies in flight and queues of products, in any order the rules allow."""

    def __init__(self, rng, left_out):
        self.rng, self.left_out = rng, left_out
        self.roles, self.copies, self.queues = {}, [], {}

    def copy(self, land):
        self.copies.append(land)

    def issue(self, queue, done):
        self.queues.setdefault(queue, []).append(done)

    def wait(self, name, bar, phase):
        """What a role yields; a wait that is left out lets it pass."""
        return None if name == self.left_out else (bar, phase)

    def run(self):
        speed = {}
        pace = lambda k: speed.setdefault(k, self.rng.choice([0.02, 0.2, 1, 5]))  # noqa: E731
        waits = {}
        while self.roles:
            acts = [("queue", k) for k, v in self.queues.items() if v]
            acts += [("copy", k) for k in range(len(self.copies))]
            for name in self.roles:
                if waits.get(name) is None:
                    acts.append(("role", name))
                    continue
                bar, phase = waits[name]
                assert bar.phase <= phase + 1, f"{name} missed phase {phase}"
                if bar.phase == phase + 1:
                    acts.append(("role", name))
            assert acts, "nobody can go on"
            kind, which = self.rng.choices(
                acts, [pace("copy" if k == "copy" else w) for k, w in acts])[0]
            if kind == "queue":
                self.queues[which].pop(0)()
            elif kind == "copy":
                self.copies.pop(which)()
            else:
                try:
                    waits[which] = next(self.roles[which])
                except StopIteration:
                    del self.roles[which]


def few_rows(rng, left_out=None):
    """paged_attn.cu: loader, rotation, QK, PV, softmax in two halves of the rows."""
    m = Machine(rng, left_out)
    rope = rng.random() < 0.7
    units = [rng.choice([1, 1, 1, 2, 3, 4]) for _ in range(rng.randint(1, 8))]
    blocks = [(i, b) for i, nb in enumerate(units) for b in range(nb)]
    q_full, q_free, q_turned = Bar(), Bar(), Bar()
    kv_full, kv_free = [Bar() for _ in range(4)], [Bar() for _ in range(4)]
    x_full, s_free = [Bar(), Bar()], [Bar(4), Bar(4)]
    s_full, p_full, o_full, o_free = Bar(2), Bar(4), Bar(), Bar(4)
    group = [Bar(2), Bar(2)]
    tile, x, S, pages = [None] * 4, [None] * 2, [None] * 2, [None] * 2
    at = dict(q=None, turned=None, O=None)
    P = {}

    def put(to, k, v, *bars):
        def land():
            to[k] = v
            for b in bars:
                b.arrive()
        return land

    def loader():
        for g in range(len(blocks)):
            pages[g & 1] = g
            x[g & 1] = None
            m.copy(put(x, g & 1, g, x_full[g & 1]))
            for c in range(4):
                yield m.wait("kv_free", kv_free[c], g - 1)
                tile[c] = None
                m.copy(put(tile, c, g, kv_full[c]))
            yield None

    def turn():
        for i in range(len(units)):
            yield q_full, i
            assert at["q"] == i
            at["turned"] = i
            q_turned.arrive()

    def qk():
        g = 0
        for i, nb in enumerate(units):
            yield m.wait("q_free", q_free, i - 1)
            at["q"] = None
            m.copy(put(at, "q", i, q_full))
            yield q_full, i
            for b in range(nb):
                yield m.wait("s_free", s_free[g & 1], (g >> 1) - 1)
                yield m.wait("x_full", x_full[g & 1], g >> 1)

                def first(i=i, g=g):
                    assert x[g & 1] == g and at["q"] == i
                    S[g & 1] = None
                m.issue("qk", first)
                for c in range(4):
                    yield m.wait("kv_full", kv_full[c], g)
                    if c == 2 and b == 0 and rope:
                        yield m.wait("q_turned", q_turned, i)

                    def step(i=i, g=g, c=c, last=b == nb - 1):
                        assert tile[c] == g and at["q"] == i
                        assert c < 2 or not rope or at["turned"] == i
                        if c == 3:
                            S[g & 1] = g
                            s_full.arrive()
                            if last:
                                q_free.arrive()
                    m.issue("qk", step)
                g += 1

    def pv():
        s_full.arrive()
        g = 0
        for i, nb in enumerate(units):
            for b in range(nb):
                yield p_full, g
                if b == 0 and i > 0:
                    yield m.wait("o_free", o_free, i - 1)
                for c in range(4):
                    def step(i=i, g=g, b=b, c=c, last=b == nb - 1):
                        assert tile[c] == g and (c < 3 or x[g & 1] == g)
                        assert list(P.values()) == [g] * 4
                        at["O"] = (i, b, c)
                        kv_free[c].arrive()
                        if c == 3:
                            s_full.arrive()
                            if last:
                                o_full.arrive()
                    m.issue("pv", step)
                g += 1

    def softmax(half, w):
        g = syncs = 0
        for i, nb in enumerate(units):
            for b in range(nb):
                yield s_full, g
                yield x_full[g & 1], g >> 1
                assert S[g & 1] == g and pages[g & 1] == g
                yield None
                assert S[g & 1] == g
                s_free[g & 1].arrive()
                group[half].arrive()          # the vote on a new maximum
                yield group[half], syncs
                syncs += 1
                assert b == 0 or at["O"] == (i, b - 1, 3)   # it may be rescaled here
                P[half, w] = g
                p_full.arrive()
                yield None
                g += 1
            yield o_full, i
            for _ in range(4):
                assert at["O"] == (i, nb - 1, 3)
                yield None
            o_free.arrive()

    m.roles = dict(load=loader(), qk=qk(), pv=pv())
    if rope:
        m.roles["turn"] = turn()
    for half in range(2):
        for w in range(2):
            P[half, w] = None
            m.roles["soft", half, w] = softmax(half, w)
    return m


def chunk(rng, left_out=None):
    """paged_chunk.cu: loader, queries, products by one warp, softmax, stores."""
    m = Machine(rng, left_out)
    part, units = rng.randint(0, 1), []
    for _ in range(rng.randint(1, 9)):
        units.append((part, rng.choice([1, 1, 1, 2, 3])))
        part ^= 1
    n = len(units)
    fresh = [i == 0 or units[i][0] == 0 for i in range(n)]
    last_of_q = [units[i][0] == 1 or i == n - 1 for i in range(n)]
    blocks = [(i, b) for i, (_, nb) in enumerate(units) for b in range(nb)]
    full, f_free, v_free = ([Bar() for _ in range(4)] for _ in range(3))
    pg_full, o_free = [Bar(), Bar()], [Bar(2), Bar(2)]
    q_full, q_tm, q_free = Bar(), Bar(4), Bar()
    s_full, s_free, p_full, pv_done = Bar(), Bar(4), Bar(4), Bar()
    o_full, stat_full, stat_free = Bar(), Bar(2), Bar(2)
    pair = [Bar(2), Bar(2)]
    slab, pages, sums = [None] * 4, [None] * 2, [None] * 2
    at = dict(q=None, S=None)
    O = [None, None]   # noqa: E741
    P, tm = {}, {}

    def loader():
        for g in range(len(blocks)):
            par, use = g & 1, g >> 1
            for step in range(4):
                k = 2 * par + (step & 1)
                if step < 2:
                    yield m.wait("v_free", v_free[k], use - 1)
                else:
                    yield m.wait("f_free", f_free[k], use)
                if step == 0:
                    pages[par] = g
                    pg_full[par].arrive()
                slab[k] = None

                def land(k=k, v=(g, step // 2)):
                    slab[k] = v
                    full[k].arrive()
                m.copy(land)
            yield None

    def queries():
        loads = 0
        for i in range(n):
            if not fresh[i]:
                continue
            yield m.wait("q_free", q_free, loads - 1)
            at["q"] = None

            def land(v=loads):
                at["q"] = v
                q_full.arrive()
            m.copy(land)
            loads += 1

    def products():
        g = loads = ends = i = b = 0
        pend = pend_first = pend_last = False
        wait_q = True
        while i < n or pend:
            qk = i < n and not (wait_q and pend)
            if qk:
                if wait_q:
                    yield m.wait("q_full", q_full, loads)
                    loads += 1
                    wait_q = False
                yield m.wait("s_free", s_free, g - 1)
            for half in range(2):
                if qk:
                    for h in range(2):
                        k = 2 * (g & 1) + h
                        yield m.wait("full", full[k], 2 * (g >> 1) + half)
                        use_tm = h == 1 and half ^ units[i][0]
                        if use_tm:
                            yield m.wait("q_tm", q_tm, loads - 1)

                        def step(k=k, g=g, half=half, q=loads - 1, use_tm=use_tm):
                            assert slab[k] == (g, half) and at["q"] == q
                            assert not use_tm or list(tm.values()) == [q] * 4
                            at["S"] = None
                            if half == 0:
                                f_free[k].arrive()
                        m.issue("mma", step)

                    def whole(g=g, last=b == units[i][1] - 1 and last_of_q[i]):
                        at["S"] = g
                        s_full.arrive()
                        if last:
                            q_free.arrive()
                    if half == 1:
                        m.issue("mma", whole)
                if pend:
                    if half == 0:
                        yield m.wait("p_full", p_full, g - 1)
                    if pend_first and ends > 0:
                        yield m.wait("o_free", o_free[half], ends - 1)

                    def pv(g=g - 1, half=half, u=ends, last=pend_last):
                        k = 2 * (g & 1) + half
                        assert slab[k] == (g, 1) and list(P.values()) == [g] * 4
                        O[half] = (u, g)
                        v_free[k].arrive()
                        if half == 1:
                            pv_done.arrive()
                            if last:
                                o_full.arrive()
                    m.issue("mma", pv)
            if pend and pend_last:
                ends += 1
            pend = qk
            if qk:
                pend_first, pend_last = b == 0, b == units[i][1] - 1
                g += 1
                b += 1
                if b == units[i][1]:
                    b, i = 0, i + 1
                    wait_q = i < n and units[i][0] == 0

    def softmax(sp, hh):
        g = loads = syncs = 0
        for i, (_, nb) in enumerate(units):
            if fresh[i]:
                tm[sp, hh] = loads
                loads += 1
                yield None
                q_tm.arrive()
            for b in range(nb):
                yield m.wait("s_full", s_full, g)
                yield pg_full[g & 1], g >> 1
                assert at["S"] == g and pages[g & 1] == g
                yield None
                assert at["S"] == g
                s_free.arrive()
                pair[sp].arrive()             # the vote on a new maximum
                yield pair[sp], syncs
                syncs += 1
                yield m.wait("pv_done", pv_done, g - 1)
                assert b == 0 or O[hh] == (i, g - 1)        # it may be rescaled here
                P[sp, hh] = g
                p_full.arrive()
                yield None
                g += 1
            pair[sp].arrive()
            yield pair[sp], syncs
            syncs += 1
            if hh == 0:
                if i > 0:
                    yield m.wait("stat_free", stat_free, i - 1)
                sums[sp] = i
                stat_full.arrive()
                yield None

    def stores(sp):
        g = -1
        for i, (_, nb) in enumerate(units):
            g += nb
            yield stat_full, i
            assert sums[sp] == i
            stat_free.arrive()
            yield o_full, i
            for half in range(2):
                for _ in range(2):
                    assert O[half] == (i, g)
                    yield None
                o_free[half].arrive()

    m.roles = dict(load=loader(), q=queries(), mma=products())
    for sp in range(2):
        m.roles["out", sp] = stores(sp)
        for hh in range(2):
            P[sp, hh] = tm[sp, hh] = None
            m.roles["soft", sp, hh] = softmax(sp, hh)
    return m


@pytest.mark.parametrize("kernel", [few_rows, chunk])
def test_protocol_holds_in_random_schedules(kernel):
    rng = random.Random(12)
    for _ in range(800):
        kernel(rng).run()


@pytest.mark.parametrize("kernel,left_out", [
    (few_rows, w) for w in ("kv_free", "kv_full", "x_full", "q_free", "q_turned")] + [
    (chunk, w) for w in ("v_free", "f_free", "full", "q_free", "q_full", "q_tm", "s_free", "s_full",
                         "p_full", "pv_done", "o_free", "stat_free")])
def test_a_wait_that_is_missing_is_found(kernel, left_out):
    rng = random.Random(13)
    for _ in range(400):
        try:
            kernel(rng, left_out).run()
        except AssertionError:
            return
    pytest.fail(f"400 schedules without {left_out} went well")
