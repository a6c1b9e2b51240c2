"""Model check of the backward kernels' barrier protocol (csrc/bwd_sm103.cu), on the CPU.

The producers, the copy engine (loads that land at any later time), the MMA issuer, an in-order tensor pipe and the warps
that compute run as coroutines under random schedules.  mbarriers count arrivals and pending bytes as the hardware does: a waiter sees only
the parity of a completed phase, and an arrival at a phase that has all its arrivals is an error (on the GPU, a fault).  The
model checks that every product reads the tiles and the values that it is meant to, that nothing is overwritten before its
last reader is done, and that the run ends with nothing in flight.  Planted mistakes (a wait left out) have to be found.
"""
import random

import pytest

# dS and dQ or dK; dV; lse of the streamed rows; operands in tensor memory; score buffers; ring slots; slots through which the first
# resident operand comes (0: a buffer of its own)
MODES = {
    "q64": dict(ds=1, dv=0, vec=0, a1t=1, a2t=1, nsb=2, slots=8), "q128": dict(ds=1, dv=0, vec=0, a1t=1, a2t=1, nsb=1, slots=5),
    "q256": dict(ds=1, dv=0, vec=0, a1t=1, a2t=0, nsb=1, slots=5, ring=2), "kv64": dict(ds=1, dv=1, vec=1, a1t=0, a2t=0, nsb=2, slots=8),
    "kv128": dict(ds=1, dv=1, vec=1, a1t=0, a2t=0, nsb=1, slots=5), "k256": dict(ds=1, dv=0, vec=1, a1t=1, a2t=0, nsb=1, slots=5, ring=2),
    "v256": dict(ds=0, dv=1, vec=1, a1t=1, a2t=0, nsb=2, slots=7, ring=2),
}
WARPS = 3


class Violation(Exception):
    pass


def need(ok, what):
    if not ok:
        raise Violation(what)


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def arrive(self, tx=0):
        need(self.pending > 0, "arrival at a phase that has all its arrivals")
        self.pending -= 1
        self.tx += tx
        self._turn()

    def land(self, tx):
        self.tx -= tx
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


def simulate(mode, seed, leave_out=None):
    m, rnd = dict(dict(ring=0), **MODES[mode]), random.Random(seed)
    buffers = ([] if m["ring"] else [0]) + ([1] if m["ds"] else [])   # of the resident operands
    units = [rnd.choice((1, 1, 2, 3, 5)) for _ in range(rnd.randint(1, 5))]
    N, nsb = m["slots"], m["nsb"]
    full, empty = [Bar(1) for _ in range(N)], [Bar(1) for _ in range(N)]
    res, free, acc = [Bar(1), Bar(1)], [Bar(1), Bar(1)], Bar(1)
    bar_s, bar_p = [Bar(1), Bar(1)], [Bar(WARPS), Bar(WARPS)]
    dp, ds = Bar(1), Bar(WARPS)
    vec, vec_free = [Bar(1), Bar(1)], [Bar(WARPS), Bar(WARPS)]
    slot, resident, operand, vecs = [None] * N, [None, None], [None, None], [None, None]    # what memory holds
    landing, pipe = [], []
    scores, grads = [None, None], [None]           # ("s", g), or per warp ("p", g) written over it
    p_by = [set(), set()]
    ds_by = set()
    sums = {"acc": [], "accv": []}
    got = []

    def wait(bar, parity, name=None):
        while name != leave_out and not bar.passed(parity):
            yield
        yield

    def ring():
        use = 0
        for u, n in enumerate(units):
            for what in [("r", u, i) for i in range(m["ring"])] + [(i, sum(units[:u]) + j) for j in range(n) for i in (0, 1)]:
                s = use % N
                yield from wait(empty[s], ((use // N) & 1) ^ 1, "empty")
                full[s].arrive(1)
                slot[s] = None
                landing.append((slot, s, what, full[s]))
                use += 1
                yield

    def second():
        g = 0
        for u, n in enumerate(units):
            for i in buffers:
                if u:
                    yield from wait(free[i], (u - 1) & 1, f"free{i}")
                res[i].arrive(1)
                resident[i] = None
                landing.append((resident, i, u, res[i]))
                yield
            for j in range(n if m["vec"] else 0):
                v = g & 1
                yield from wait(vec_free[v], ((g >> 1) & 1) ^ 1, "vec_free")
                vec[v].arrive(1)
                vecs[v] = None
                landing.append((vecs, v, g, vec[v]))
                g += 1
                yield

    def engine():
        while True:
            if landing and rnd.random() < 0.3:
                where, i, what, bar = landing.pop(rnd.randrange(len(landing)))
                where[i] = what
                bar.land(1)
            yield

    def tensor():
        while True:
            if pipe and rnd.random() < 0.5:
                pipe.pop(0)()
            yield

    def mma():
        g = use = 0

        def op_s(u, gs, x):
            def f():
                need(slot[x % N] == (0, gs), "scores read another tile")
                need((operand[0] if m["a1t"] else resident[0]) == u, "scores read another resident tile")
                b = gs % nsb
                need(scores[b] is None or (scores[b][0] == "free" and len(p_by[b]) in (0, WARPS)), "scores written over values in use")
                scores[b], p_by[b] = ("s", gs), set()
            return f

        def op_dp(u, gs, x):
            def f():
                need(slot[(x + 1) % N] == (1, gs), "dP reads another tile")
                need((operand[1] if m["a2t"] else resident[1]) == u, "dP reads another resident tile")
                need(grads[0] is None or grads[0][0] == "free", "dP written over values in use")
                grads[0] = ("dp", gs)
                ds_by.clear()
            return f

        def op_dv(u, gs, x, first):
            def f():
                b = gs % nsb
                need(slot[(x + 1) % N] == (1, gs), "dV reads another tile")
                need(p_by[b] == set(range(WARPS)) and scores[b] == ("s", gs), "dV reads values that are not P")
                scores[b] = ("free", gs)
                if first:
                    need(not sums["accv"], "dV begun over a sum in use")
                sums["accv"].append(gs)
            return f

        def op_acc(u, gs, x, first):
            def f():
                need(slot[x % N] == (0, gs), "dQ or dK reads another tile")
                need(ds_by == set(range(WARPS)) and grads[0] == ("dp", gs), "dQ or dK reads values that are not dS")
                grads[0] = ("free", gs)
                if first:
                    need(not sums["acc"], "dQ or dK begun over a sum in use")
                sums["acc"].append(gs)
            return f

        commit = lambda bar: pipe.append(bar.arrive)  # noqa: E731
        full_of = lambda use, name: wait(full[use % N], (use // N) & 1, name)  # noqa: E731

        def do_s(u, gs, x, last):
            yield from full_of(x, "full1")
            pipe.append(op_s(u, gs, x))
            commit(bar_s[gs & 1])
            if not m["ds"]:
                commit(empty[x % N])
            if last and not m["a1t"]:
                commit(free[0])

        def do_dp(u, gs, x, last):
            yield from full_of(x + 1, "full2")
            pipe.append(op_dp(u, gs, x))
            commit(dp)
            if not m["dv"]:
                commit(empty[(x + 1) % N])
            if last and not m["a2t"]:
                commit(free[1])

        for u, n in enumerate(units):
            if not m["ring"]:
                yield from wait(res[0], u & 1, "res0")
            if m["a2t"]:
                yield from wait(res[1], u & 1, "res1")
            for i in range(m["ring"]):
                yield from full_of(use, "full_r")

                def copy_slot(u=u, i=i, use=use):
                    need(slot[use % N] == ("r", u, i), "another tile is copied")
                    operand[0] = u if i == m["ring"] - 1 else None
                pipe.append(copy_slot)
                commit(empty[use % N])
                use += 1
            if m["a1t"] and not m["ring"]:
                def copy(i, u=u):
                    need(resident[i] == u, "another resident tile is copied")
                    operand[i] = u
                pipe.append(lambda copy=copy: copy(0))
                commit(free[0])
                if m["a2t"]:
                    pipe.append(lambda copy=copy: copy(1))
                    commit(free[1])
            yield from do_s(u, g, use, n == 1)
            if m["ds"]:
                if not m["a2t"]:
                    yield from wait(res[1], u & 1, "res1")
                yield from do_dp(u, g, use, n == 1)
            for j in range(n):
                gs, more = g + j, j + 1 < n
                if nsb == 2 and more:
                    yield from do_s(u, gs + 1, use + 2, j + 2 == n)
                yield from wait(bar_p[gs & 1], (gs >> 1) & 1, "p")
                if m["dv"]:
                    if not m["ds"]:
                        yield from full_of(use + 1, "full2")
                    pipe.append(op_dv(u, gs, use, j == 0))
                    commit(empty[(use + 1) % N])
                if nsb == 1 and more:
                    yield from do_s(u, gs + 1, use + 2, j + 2 == n)
                if m["ds"]:
                    yield from wait(ds, gs & 1, "ds")
                    pipe.append(op_acc(u, gs, use, j == 0))
                    commit(empty[use % N])
                    if more:
                        yield from do_dp(u, gs + 1, use + 2, j + 2 == n)
                use += 2
            commit(acc)
            g += n
        yield from wait(acc, (len(units) - 1) & 1)

    def compute(w):
        g = 0
        for u, n in enumerate(units):
            for j in range(n):
                gs = g + j
                b = gs % nsb
                if m["vec"]:
                    yield from wait(vec[gs & 1], (gs >> 1) & 1, "vec")
                yield from wait(bar_s[gs & 1], (gs >> 1) & 1, "s")
                need(scores[b] == ("s", gs) and w not in p_by[b], "other scores are read")
                need(not m["vec"] or vecs[gs & 1] == gs, "another tile's lse is read")
                yield
                need(scores[b] == ("s", gs), "scores changed while they are read")
                p_by[b].add(w)
                if not m["dv"] and len(p_by[b]) == WARPS:
                    scores[b] = ("free", gs)
                bar_p[gs & 1].arrive()
                yield
                if m["ds"]:
                    yield from wait(dp, gs & 1, "dp")
                    need(grads[0] == ("dp", gs) and w not in ds_by, "another dP is read")
                    need(not m["vec"] or vecs[gs & 1] == gs, "another tile's delta is read")
                    yield
                    ds_by.add(w)
                    ds.arrive()
                if m["vec"]:
                    vec_free[gs & 1].arrive()
                yield
            yield from wait(acc, u & 1, "acc")
            steps = list(range(g, g + n))
            need((not m["ds"] or sums["acc"] == steps) and (not m["dv"] or sums["accv"] == steps), "a result is read before it is whole")
            got.append((w, u))
            yield
            if sum(1 for x in got if x[1] == u) == WARPS:
                sums["acc"], sums["accv"] = [], []
            else:   # the others may still read; the next unit's first sum needs everyone's P or dS anyway
                while sum(1 for x in got if x[1] == u) < WARPS:
                    yield
            g += n

    roles = [ring(), second(), mma()] + [compute(w) for w in range(WARPS)]
    machines = [engine(), tensor()]
    speed = {id(r): rnd.choice((1, 10, 10, 100)) for r in roles + machines}   # some lag behind, some run ahead
    for _ in range(400000):
        if not roles:
            break
        r, = rnd.choices(roles + machines, [speed[id(x)] for x in roles + machines])
        try:
            next(r)
        except StopIteration:
            roles.remove(r)
    need(not roles, "the run does not end")
    while pipe:
        pipe.pop(0)()
    need(not landing, "a load is in flight at the end")
    need(len(got) == WARPS * len(units), "a result is missing")


@pytest.mark.parametrize("mode", MODES)
def test_protocol(mode):
    for seed in range(60):
        simulate(mode, seed)


# what each mode waits for, and what goes wrong without
@pytest.mark.parametrize("mode,name", [(m, n) for m, c in MODES.items() for n in ("full1", "full2", "empty", "s", "acc") +
                                       (("full_r",) if c.get("ring") else ()) + (("res1", "free1") if c["ds"] else ()) + (() if c.get("ring") else ("res0", "free0")) +
                                       (("p",) if c["dv"] or c["nsb"] == 1 else ()) +   # else implied by the wait for dS
                                       (("dp", "ds") if c["ds"] else ()) + (("vec", "vec_free") if c["vec"] else ())])
def test_a_wait_left_out_is_found(mode, name):
    for seed in range(200):
        try:
            simulate(mode, seed, name)
        except Violation:
            return
    raise AssertionError(f"{mode} without the wait for {name}: not found")
