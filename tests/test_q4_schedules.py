"""The barrier protocol of the 4-bit paged attention, run through random schedules on the CPU, as in
test_paged_schedules.py (whose machine and rules it uses): every wait is checked for missed phases
and for phases it would take for an earlier one, every buffer for whom it is for.

The four warps of a half of the unpackers are two here, as are those of a half of the softmax.
(The wait for o_free is implied by others: PV of a unit's first block waits for the P of warps that
have stored the unit before.)"""
import random

import pytest
from test_paged_schedules import Bar, Machine

RING = 4


def ahead(name, role):
    """A role whose waits never begin two phases early: by parity they would end at once."""
    for wait in role:
        assert wait is None or wait[0].phase >= wait[1], f"{name} waits ahead for phase {wait[1]}"
        yield wait


def q4(rng, left_out=None):
    """q4_attn.cu: raw loader, queries and chunk 7, QK, PV, unpackers and softmax in halves."""
    m = Machine(rng, left_out)
    rope = rng.random() < 0.7
    units = [rng.choice([1, 1, 1, 2, 3, 5]) for _ in range(rng.randint(1, 7))]
    blocks = [(i, b) for i, nb in enumerate(units) for b in range(nb)]
    n = len(blocks)
    tm_full, v_full = [Bar(4) for _ in range(3)], [Bar(4) for _ in range(3)]
    v_free = [Bar() for _ in range(4)]
    raw_free = [Bar(4) for _ in range(4)]
    raw_full = [Bar() for _ in range(4)]
    k6_full, r_full, qa_done = Bar(4), Bar(), Bar()
    q_full, q_free, q_turned = Bar(), Bar(), Bar()
    s_full, s_free, p_full, pv_done, o_full, o_free = Bar(), Bar(4), Bar(4), Bar(), Bar(), Bar(4)
    group = [Bar(2), Bar(2)]
    raw, valid = [None, None], [None] * RING      # raw: (block, part)
    tmem = {(m_, h, w): None for m_ in range(3) for h in range(2) for w in range(2)}
    V, k6 = dict(tmem), {(h, w): None for h in range(2) for w in range(2)}
    pair = lambda of, k: [of[k, h, w] for h in range(2) for w in range(2)]  # noqa: E731
    at = dict(q=None, turned=None, S=None, O=None, r=None)
    P = {}

    def loader():
        for t in range(n + 1):
            for j in range(4):
                # (the part before in the slot)
                yield m.wait("raw_free", raw_free[j ^ 2], t - (j < 2))
                if j == 0:
                    valid[t % RING] = t if t < n else "end"
                    if t == n:
                        raw_full[0].arrive()
                        return
                raw[j & 1] = None

                def land(t=t, j=j):
                    raw[j & 1] = (t, j)
                    raw_full[j].arrive()
                m.copy(land)
                yield None

    def queries():
        t = 0
        for i, nb in enumerate(units):
            yield m.wait("q_free", q_free, i - 1)
            at["q"] = None

            def land(i=i):
                at["q"] = i
                q_full.arrive()
            m.copy(land)
            for b in range(nb):
                yield m.wait("v_free of chunk 7", v_free[3], t - 1)
                at["r"] = None

                def rope_land(t=t):
                    at["r"] = t
                    r_full.arrive()
                m.copy(rope_land)
                t += 1
                if b == 0 and rope:
                    yield q_full, i
                    assert at["q"] == i
                    at["turned"] = i
                    q_turned.arrive()

    def qk():
        g = 0
        for i, nb in enumerate(units):
            yield m.wait("q_full", q_full, i)
            for b in range(nb):
                yield m.wait("s_free", s_free, g - 1)
                for h in range(3):
                    yield m.wait("tm_full", tm_full[h], g)

                    def step(i=i, g=g, h=h):
                        assert at["q"] == i and pair(tmem, h) == [g] * 4
                        at["S"] = None
                        if h == 2:
                            qa_done.arrive()
                    m.issue("qk", step)
                yield m.wait("k6_full", k6_full, g)
                yield m.wait("r_full", r_full, g)
                if b == 0 and rope:
                    yield m.wait("q_turned", q_turned, i)

                def whole(i=i, g=g, last=b == nb - 1):
                    assert at["q"] == i and list(k6.values()) == [g] * 4 and at["r"] == g
                    assert not rope or at["turned"] == i
                    at["S"] = g
                    s_full.arrive()
                    if last:
                        q_free.arrive()
                m.issue("qk", whole)
                g += 1

    def pv():
        g = 0
        for i, nb in enumerate(units):
            for b in range(nb):
                yield p_full, g
                if b == 0 and i > 0:
                    yield m.wait("o_free", o_free, i - 1)
                for st in range(4):
                    h = (st + 3) & 3
                    if st:
                        yield m.wait("v_full", v_full[h], g)

                    def step(i=i, g=g, b=b, h=h, st=st, last=b == nb - 1):
                        assert list(P.values()) == [g] * 4
                        if st == 0:
                            assert list(k6.values()) == [g] * 4 and at["r"] == g
                        else:
                            assert pair(V, h) == [g] * 4
                        at["O"] = (i, b, st)
                        v_free[h].arrive()
                        if st == 3:
                            pv_done.arrive()
                            if last:
                                o_full.arrive()
                    m.issue("pv", step)
                g += 1

    def unpack(h, w):
        have, before, t = True, False, 0
        while True:
            if before:
                if t > 1:
                    yield m.wait("v_free of chunk 6", v_free[3], t - 2)
                k6[h, w] = t - 1
                yield None
                k6_full.arrive()
            if have:
                yield m.wait("raw_full", raw_full[0], t)
                have = valid[t % RING] != "end"
            if not have and not before:
                return
            if have:
                assert raw[0] == (t, 0) and valid[t % RING] == t
                if h == 1:
                    yield None
                    raw_free[0].arrive()
            for k in range(3):
                part = k + h
                if have:
                    yield m.wait("raw_full", raw_full[part], t)
                    assert raw[part & 1] == (t, part)
                    yield None
                    assert raw[part & 1] == (t, part)
                    if part < 3:
                        raw_free[part].arrive()
                if before:
                    if t > 1:
                        yield m.wait("v_free", v_free[k], t - 2)
                    assert tmem[k, h, w] == t - 1
                    V[k, h, w] = t - 1
                    yield None
                    v_full[k].arrive()
                    if k == 0 and have:
                        yield m.wait("qa_done", qa_done, t - 1)
                if have:
                    tmem[k, h, w] = None
                    if k == 2:
                        yield m.wait("raw_full", raw_full[3], t)
                        assert raw[1] == (t, 3)
                        yield None
                        raw_free[3].arrive()
                    tmem[k, h, w] = t
                    yield None
                    tm_full[k].arrive()
            before = have
            t += 1

    def softmax(half, w):
        g = syncs = 0
        for i, nb in enumerate(units):
            for b in range(nb):
                yield m.wait("s_full", s_full, g)
                yield k6_full, g
                assert at["S"] == g and valid[g % RING] == g
                yield None
                assert at["S"] == g
                s_free.arrive()
                group[half].arrive()          # the vote on a new maximum
                yield group[half], syncs
                syncs += 1
                yield m.wait("pv_done", pv_done, g - 1)
                assert b == 0 or at["O"] == (i, b - 1, 3)   # it may be rescaled here
                P[half, w] = g
                yield None
                p_full.arrive()
                g += 1
            yield o_full, i
            for _ in range(3):
                assert at["O"] == (i, nb - 1, 3)
                yield None
            o_free.arrive()

    m.roles = dict(load=loader(), q=queries(), qk=qk(), pv=pv())
    for half in range(2):
        for w in range(2):
            m.roles["unpack", half, w] = unpack(half, w)
            P[half, w] = None
            m.roles["soft", half, w] = softmax(half, w)
    m.roles = {k: ahead(k, v) for k, v in m.roles.items()}
    return m


def test_protocol_holds_in_random_schedules():
    rng = random.Random(12)
    for _ in range(800):
        q4(rng).run()


@pytest.mark.parametrize("left_out", ["raw_free", "raw_full", "v_free", "v_free of chunk 6",
                                      "v_free of chunk 7", "tm_full", "qa_done", "v_full", "k6_full",
                                      "r_full", "q_free", "q_full", "q_turned", "s_free", "s_full",
                                      "pv_done"])
def test_a_wait_that_is_missing_is_found(left_out):
    rng = random.Random(13)
    for _ in range(400):
        try:
            q4(rng, left_out).run()
        except AssertionError:
            return
    pytest.fail(f"400 schedules without {left_out} went well")
