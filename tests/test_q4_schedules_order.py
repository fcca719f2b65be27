"""The barrier protocol of the 4-bit paged attention in random schedules, step by step in the kernel's
own order: the loader writes the list of a block's keys before it waits for a slot; softmax warps
clean chunks 6 and 7 in place, rescale O^T at a new maximum, hand maxima and sums to their half's
first warp, which walks a segment ahead. (test_q4_schedules.py has the same roles
with a stricter loader and without these steps; the machine and its rules are
test_paged_schedules.py's.)

Every wait is left out once, in the model. Those of MUST_FAIL have to be found by some schedule. Those
of IMPLIED never are: other waits imply their order. The kernel has them all the same, o_free as a
guard, the softmax's k6_full and r_full since plain accesses follow to what other warps and copies
wrote (QK's completion, which implies both, orders the products alone). Not in the model: the waits
for copies and products in flight at a kernel's end."""
import random

import pytest
from test_paged_schedules import Bar, Machine

MUST_FAIL = ["raw_free", "raw_full", "v_free", "v_free of chunk 6", "v_free of chunk 7", "tm_full",
             "qa_done", "v_full", "k6_full", "r_full", "q_free", "q_full", "q_full of the turn",
             "q_turned", "s_free", "s_full", "p_full", "pv_done", "pv_done of the rescale", "o_full",
             "group"]
IMPLIED = ["o_free", "k6_full of the softmax", "r_full of the cleaning"]


def ahead(name, role):
    """A role whose waits never begin two phases early: by parity they would end at once."""
    for wait in role:
        assert wait is None or wait[0].phase >= wait[1], f"{name} waits ahead for phase {wait[1]}"
        yield wait


class Tiles:
    """What the roles share, and the block (or unit) that each place is for."""

    def __init__(self, ring):
        four = [(h, w) for h in range(2) for w in range(2)]
        self.raw = [None, None]                                  # (block, part)
        self.valid = [None] * ring                               # a block's keys, or "end"
        self.tmem = {(m, *k): None for m in range(3) for k in four}
        self.v = dict(self.tmem)
        self.k6 = {k: None for k in four}                        # by half of the dims, keys
        self.clean = [None, None]                                # keys made finite in 6 and 7
        self.rope = self.q = self.turned = self.s = self.o = None
        self.p = {k: None for k in four}                         # by half of the rows, keys
        self.red = {k: None for k in four}
        self.factor = [None, None]                               # alpha, then 1 / sum
        self.segment = [[None, None], [None, None]]

    def pair(self, of, m):
        return [of[m, h, w] for h in range(2) for w in range(2)]


def q4(rng, left_out=None, ring=4):
    m = Machine(rng, left_out)
    x = Tiles(ring)
    rope = rng.random() < 0.7
    units = [rng.choice([1, 1, 1, 2, 3, 5]) for _ in range(rng.randint(1, 7))]
    blocks = [(i, b, b == nb - 1) for i, nb in enumerate(units) for b in range(nb)]
    n = len(blocks)
    often = rng.choice([0.1, 0.5, 0.9])
    dirty = [[rng.random() < often for _ in range(2)] for _ in range(n)]      # by keys
    rises = [[rng.random() < often for _ in range(2)] for _ in range(n)]      # by half of the rows
    tm_full, v_full = [Bar(4) for _ in range(3)], [Bar(4) for _ in range(3)]
    v_free, raw_free = [Bar() for _ in range(4)], [Bar(4) for _ in range(4)]
    raw_full = [Bar() for _ in range(4)]
    k6_full, r_full, qa_done = Bar(4), Bar(), Bar()
    q_full, q_free, q_turned = Bar(), Bar(), Bar()
    s_full, s_free, p_full, pv_done = Bar(), Bar(4), Bar(4), Bar()
    o_full, o_free, group = Bar(), Bar(4), [Bar(2), Bar(2)]

    def loader():
        for t in range(n + 1):
            x.valid[t % ring] = t if t < n else "end"
            yield None
            for j in range(4):
                # (the part before in the slot)
                yield m.wait("raw_free", raw_free[j ^ 2], t - (j < 2))
                if t == n:
                    raw_full[0].arrive()
                    return
                x.raw[j & 1] = None

                def land(t=t, j=j):
                    x.raw[j & 1] = (t, j)
                    raw_full[j].arrive()
                m.copy(land)

    def queries():
        for t, (i, b, _) in enumerate(blocks):
            if b == 0:
                yield m.wait("q_free", q_free, i - 1)
                x.q = None

                def land(i=i):
                    x.q = i
                    q_full.arrive()
                m.copy(land)
            if t > 0:
                yield m.wait("v_free of chunk 7", v_free[3], t - 1)
            x.rope = None

            def rope_land(t=t):
                x.rope = t
                r_full.arrive()
            m.copy(rope_land)
            if b == 0 and rope:
                yield m.wait("q_full of the turn", q_full, i)
                assert x.q == i
                yield None
                x.turned = i
                q_turned.arrive()

    def qk():
        for g, (i, b, last) in enumerate(blocks):
            if b == 0:
                yield m.wait("q_full", q_full, i)
            yield m.wait("s_free", s_free, g - 1)
            for k in range(3):
                yield m.wait("tm_full", tm_full[k], g)

                def step(i=i, g=g, k=k):
                    assert x.q == i and x.pair(x.tmem, k) == [g] * 4
                    x.s = None
                    if k == 2:
                        qa_done.arrive()
                m.issue("qk", step)
            yield m.wait("k6_full", k6_full, g)
            yield m.wait("r_full", r_full, g)
            if b == 0 and rope:
                yield m.wait("q_turned", q_turned, i)

            def whole(i=i, g=g, last=last):
                assert x.q == i and list(x.k6.values()) == [g] * 4 and x.rope == g
                assert not rope or x.turned == i
                x.s = g
                s_full.arrive()
                if last:
                    q_free.arrive()
            m.issue("qk", whole)

    def pv():
        for g, (i, b, last) in enumerate(blocks):
            yield m.wait("p_full", p_full, g)
            if b == 0 and i > 0:
                yield m.wait("o_free", o_free, i - 1)
            for st in range(4):
                k = (st + 3) & 3
                if st:
                    yield m.wait("v_full", v_full[k], g)

                def step(i=i, g=g, b=b, k=k, st=st, last=last):
                    assert list(x.p.values()) == [g] * 4
                    if st == 0:
                        assert list(x.k6.values()) == [g] * 4 and x.rope == g
                        assert all(x.clean[w] == g for w in range(2) if dirty[g][w])
                    else:
                        assert x.pair(x.v, k) == [g] * 4
                    x.o = (i, b, st)
                    v_free[k].arrive()
                    if st == 3:
                        pv_done.arrive()
                        if last:
                            o_full.arrive()
                m.issue("pv", step)

    def unpack(h, w):
        have, before, t = True, False, 0
        while True:
            if before:
                if t > 1:
                    yield m.wait("v_free of chunk 6", v_free[3], t - 2)
                x.k6[h, w] = t - 1
                yield None
                k6_full.arrive()
            if have:
                yield m.wait("raw_full", raw_full[0], t)
                have = x.valid[t % ring] != "end"
            if not have and not before:
                return
            if have:
                assert x.raw[0] == (t, 0) and x.valid[t % ring] == t
                yield None
                assert x.raw[0] == (t, 0)
                if h == 1:
                    raw_free[0].arrive()
            for k in range(3):
                part = k + h
                if have:
                    yield m.wait("raw_full", raw_full[part], t)
                    assert x.raw[part & 1] == (t, part)
                    yield None
                    assert x.raw[part & 1] == (t, part)
                    if part < 3:
                        raw_free[part].arrive()
                if before:
                    if t > 1:
                        yield m.wait("v_free", v_free[k], t - 2)
                    assert x.tmem[k, h, w] == t - 1
                    x.v[k, h, w] = t - 1
                    yield None
                    v_full[k].arrive()
                    if k == 0 and have:
                        yield m.wait("qa_done", qa_done, t - 1)
                if have:
                    x.tmem[k, h, w] = None
                    if k == 2:
                        if h == 0:
                            yield m.wait("raw_full", raw_full[3], t)
                        assert x.raw[1] == (t, 3)
                        yield None
                        assert x.raw[1] == (t, 3)
                        raw_free[3].arrive()
                    x.tmem[k, h, w] = t
                    yield None
                    tm_full[k].arrive()
            before = have
            t += 1

    def softmax(half, w):
        syncs = 0

        def meet():
            nonlocal syncs
            group[half].arrive()
            syncs += 1
            return m.wait("group", group[half], syncs - 1)

        if w == 0:
            x.segment[half][0] = 0
        yield meet()
        g = 0
        for i, nb in enumerate(units):
            assert x.segment[half][i & 1] == i
            yield meet()
            if w == 0:
                x.segment[half][(i + 1) & 1] = i + 1
            for b in range(nb):
                assert x.segment[half][i & 1] == i
                yield m.wait("s_full", s_full, g)
                yield m.wait("k6_full of the softmax", k6_full, g)
                assert x.s == g and x.valid[g % ring] == g
                yield None
                assert x.s == g
                s_free.arrive()
                if dirty[g][w]:
                    yield m.wait("r_full of the cleaning", r_full, g)
                    for _ in range(2):
                        assert x.rope == g and [x.k6[h, w] for h in range(2)] == [g] * 2
                        yield None
                    x.clean[w] = g
                yield meet()                  # the vote on a new maximum
                if rises[g][half]:
                    x.red[half, w] = ("max", g)
                    yield meet()
                    if w == 0:
                        assert [x.red[half, k] for k in range(2)] == [("max", g)] * 2
                        x.factor[half] = ("alpha", g)
                    yield meet()
                    assert x.factor[half] == ("alpha", g)
                    if b > 0:
                        yield m.wait("pv_done of the rescale", pv_done, g - 1)
                        for _ in range(2):
                            assert x.o == (i, b - 1, 3) and x.factor[half] == ("alpha", g)
                            yield None
                yield m.wait("pv_done", pv_done, g - 1)
                x.p[half, w] = g
                yield None
                p_full.arrive()
                g += 1
            x.red[half, w] = ("sum", i)
            yield meet()
            if w == 0:
                assert [x.red[half, k] for k in range(2)] == [("sum", i)] * 2
                x.factor[half] = ("1 / sum", i)
            yield meet()
            yield m.wait("o_full", o_full, i)
            for _ in range(3):
                assert x.o == (i, nb - 1, 3) and x.factor[half] == ("1 / sum", i)
                yield None
            o_free.arrive()

    m.roles = dict(load=loader(), q=queries(), qk=qk(), pv=pv())
    for half in range(2):
        for w in range(2):
            m.roles["unpack", half, w] = unpack(half, w)
            m.roles["soft", half, w] = softmax(half, w)
    m.roles = {k: ahead(k, v) for k, v in m.roles.items()}
    return m


def test_the_kernels_order_holds_in_random_schedules():
    rng = random.Random(21)
    for _ in range(800):
        q4(rng).run()


@pytest.mark.parametrize("left_out", MUST_FAIL)
def test_a_wait_that_is_missing_is_found(left_out):
    rng = random.Random(22)
    for _ in range(600):
        try:
            q4(rng, left_out).run()
        except AssertionError:
            return
    pytest.fail(f"600 schedules without {left_out} went well")


@pytest.mark.parametrize("left_out", IMPLIED)
def test_waits_that_others_imply(left_out):
    rng = random.Random(23)
    for _ in range(300):
        q4(rng, left_out).run()


def test_lists_of_keys_for_two_blocks_are_too_few():
    """The loader writes a block's list while the softmax may read that of the block two before."""
    rng = random.Random(24)
    with pytest.raises(AssertionError):
        for _ in range(600):
            q4(rng, ring=2).run()
