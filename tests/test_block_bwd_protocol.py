"""Model of the mbarrier protocol of the whole-block attention gradient (no GPU).

The kernel (chunked_block_self_b200/csrc/block_bwd_sm100a.cu) takes (block,
head) items of one or two 128-key tiles; a tile has up to four units of 64
queries, which two elementwise groups take in turn.  One warp issues S and D,
another dV, dK and dQ; K, Q, dO and V have one or two slots each.

A parity wait on an mbarrier answers correctly only for the barrier's current
phase or the one after it.  This model replays the kernel's waits, arrivals
and commits (copies and MMAs complete at random later times, in order for each
issuing warp) under random interleavings, every wait carrying the absolute
phase it means.  It fails if a parity wait would answer differently from the
true one, or if the roles deadlock."""
import random

import pytest

K, Q, DO, V = range(4)
WARPS = 2   # of a group: enough for one to run ahead of another


class _Bar:
    def __init__(self, count):
        self.count, self.pending, self.phases = count, 0, 0

    def arrive(self):
        self.pending += 1
        assert self.pending <= self.count
        if self.pending == self.count:
            self.pending, self.phases = 0, self.phases + 1


def _slot(m, n, slots):
    """(slot, earlier uses) of matrix m of item n."""
    two = slots - 4
    twice = m < two
    return m + min(m, two) + (n & 1 if twice else 0), n >> 1 if twice else n


def _simulate(lengths, slots, seed, idle_waits=True, ds_ring=4):
    """Runs the roles over blocks of these lengths.  idle_waits: a group without
    a unit in a half waits for the half's phase before the next can end;
    ds_ring: barriers that dS is signalled on (2: one a group)."""
    rnd = random.Random(seed)
    bars, queues = {}, {"s_d": [], "products": [], "copies": []}

    def bar(name, i=0, count=1):
        return bars.setdefault((name, i), _Bar(count))

    for i in range(8):
        bar("full", i), bar("empty", i)
    for i in range(4):
        bar("ds_full", i, WARPS)
    for i in range(2):
        for name in ("ready_s", "ready_d", "s_full", "d_full", "p_empty", "dq_done"):
            bar(name, i)
        bar("cols_empty", i, 2 * WARPS), bar("s_empty", i, WARPS), bar("p_full", i, WARPS)
    bar("acc_full"), bar("acc_empty"), bar("dq_empty"), bar("idle", 0, WARPS)

    def wait(name, i, phase):
        b = bars[name, i]
        while True:
            assert (b.phases & 1 != phase & 1) == (b.phases > phase), f"parity wait on {name}{i}"
            if b.phases > phase:
                return
            yield

    def ds_bar(t):
        return (t & 3, t >> 2) if ds_ring == 4 else (t & 1, t >> 1)

    def producer():
        for n in range(len(lengths)):
            for m in (K, Q, V, DO):
                s, use = _slot(m, n, slots)
                if use > 0:
                    yield from wait("empty", s, use - 1)
                queues["copies"].append(("full", s))
                yield

    def check():
        for n in range(len(lengths)):
            if n >= 2:
                yield from wait("cols_empty", n & 1, (n >> 1) - 1)
            for name, ms in (("ready_s", (K, Q)), ("ready_d", (DO, V))):
                for m in ms:
                    yield from wait("full", *_slot(m, n, slots))
                bars[name, n & 1].arrive()
                yield

    def s_and_d():
        t = 0
        for n, L in enumerate(lengths):
            yield from wait("ready_s", n & 1, n >> 1)
            units, si = -(-L // 64) * -(-L // 128), 0
            for i in range(units):
                while si < units and si < max(i + 1, 2):
                    g, use = (t + si) & 1, (t + si) >> 1
                    if use > 0:
                        yield from wait("s_empty", g, use - 1)
                    queues["s_d"].append(("s_full", g))
                    si += 1
                    yield
                g, use = (t + i) & 1, (t + i) >> 1
                if i == 0:
                    yield from wait("ready_d", n & 1, n >> 1)
                if use > 0:
                    yield from wait("p_empty", g, use - 1)
                queues["s_d"].append(("d_full", g))
                if i + 1 == units:
                    queues["s_d"].append(("empty", _slot(V, n, slots)[0]))
                yield
            t += units

    def products():
        t = tiles = idle = 0
        commit = queues["products"].append
        for n, L in enumerate(lengths):
            for c in range(-(-L // 128)):
                if tiles > 0:
                    yield from wait("acc_empty", 0, tiles - 1)
                last_c = (c + 1) * 128 >= L
                for u in range(-(-L // 64)):
                    g, last_u = t & 1, (u + 1) * 64 >= L
                    yield from wait("p_full", g, t >> 1)
                    commit(("p_empty", g))
                    if last_u and last_c:
                        commit(("empty", _slot(DO, n, slots)[0]))
                    yield
                    yield from wait("ds_full", *ds_bar(t))
                    if idle_waits and L <= 64:
                        yield from wait("idle", 0, idle)
                        idle += 1
                    if c == 0 and (u == 1 or (u == 0 and last_u)) and n > 0:
                        yield from wait("dq_empty", 0, n - 1)
                    if last_u and last_c:
                        commit(("empty", _slot(Q, n, slots)[0]))
                    if u & 1 or last_u:
                        commit(("dq_done", u >> 1))
                    if last_u:
                        commit(("acc_full", 0))
                        if last_c:
                            commit(("empty", _slot(K, n, slots)[0]))
                    yield
                    t += 1
                tiles += 1

    def results():
        tiles = 0
        for L in lengths:
            for c in range(-(-L // 128)):
                yield from wait("acc_full", 0, tiles)
                tiles += 1
                yield
                bars["acc_empty", 0].arrive()
                if (c + 1) * 128 >= L:
                    yield
                    bars["dq_empty", 0].arrive()

    def elementwise(g):
        t, nx = 0, [0, 0]
        for n, L in enumerate(lengths):
            yield from wait("ready_s", n & 1, n >> 1)
            for _ in range(-(-L // 128)):
                u0 = (t ^ g) & 1
                for u in range(u0, -(-L // 64), 2):
                    yield from wait("s_full", g, (t + u) >> 1)
                    yield
                    bars["s_empty", g].arrive()
                    yield from wait("d_full", g, (t + u) >> 1)
                    x = u >> 1
                    if nx[x] > 0:
                        yield from wait("dq_done", x, nx[x] - 1)
                    yield
                    bars["p_full", g].arrive()
                    yield
                    if idle_waits and L > 128 and (2 + u0) * 64 >= L and nx[1] > 0:
                        yield from wait("dq_done", 1, nx[1] - 1)
                    bars["ds_full", ds_bar(t + u)[0]].arrive()
                if idle_waits:
                    if u0 * 64 >= L:
                        if nx[0] > 0:
                            yield from wait("dq_done", 0, nx[0] - 1)
                        bars["idle", 0].arrive()
                else:   # at the tile's end instead
                    if u0 * 64 >= L and nx[0] > 0:
                        yield from wait("dq_done", 0, nx[0] - 1)
                    if L > 128 and (2 + u0) * 64 >= L and nx[1] > 0:
                        yield from wait("dq_done", 1, nx[1] - 1)
                t += -(-L // 64)
                nx[0] += 1
                nx[1] += L > 128
            bars["cols_empty", n & 1].arrive()

    roles = [producer(), check(), s_and_d(), products(), results(), *(elementwise(i % 2) for i in range(2 * WARPS))]
    speed = [rnd.random() ** 2 + 0.05 for _ in roles]
    alive, quiet = list(range(len(roles))), 0
    state = None
    while alive:
        if rnd.random() < 0.3:
            ready = [q for q in queues.values() if q]
            if ready:
                bars[rnd.choice(ready).pop(0)].arrive()
        i = rnd.choices(alive, [speed[j] for j in alive])[0]
        try:
            next(roles[i])
        except StopIteration:
            alive.remove(i)
        now = (tuple((b.phases, b.pending) for b in bars.values()), len(alive))
        quiet = 0 if now != state or any(queues.values()) else quiet + 1
        state = now
        assert quiet < 2000, "deadlock"


@pytest.mark.parametrize("slots", [4, 5, 6, 7, 8])
def test_barrier_phases(slots):
    rng = random.Random(slots)
    for trial in range(120):
        top = rng.choice([64, 128, 200, 256])
        _simulate([rng.randint(1, top) for _ in range(rng.randint(1, 12))], slots, trial)


@pytest.mark.parametrize("weaker", [dict(idle_waits=False), dict(ds_ring=2)])
def test_model_catches_what_the_kernel_prevents(weaker):
    """A group without a unit that may fall behind, and one dS barrier a group,
    which the group can pass twice before the products' warp has waited once:
    the model must flag both (the same seeds pass as the kernel is)."""
    flagged = 0
    for seed in range(150):
        rng = random.Random(seed)
        lengths = [rng.randint(1, rng.choice([64, 256])) for _ in range(10)]
        _simulate(lengths, 6, seed)
        try:
            _simulate(lengths, 6, seed, **weaker)
        except AssertionError as e:
            assert "parity wait" in str(e) or "deadlock" in str(e)
            flagged += 1
    assert flagged > 0
