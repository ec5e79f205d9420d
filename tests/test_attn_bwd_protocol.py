"""Model of the mbarrier protocol of the attention gradient in tiles (no GPU).

The kernel (chunked_block_self_b200/csrc/attn_bwd_sm100a.cu) walks items of
one owner tile and T / 64 tiles of the other side: a producer with two owner
stages and a ring of eight tiles, one warp each for S, D and the accumulating
products, and two elementwise streams on alternate tiles, counted over all
items (an item of one tile leaves a stream without any).

A parity wait on an mbarrier answers correctly only for the barrier's current
phase or the one after it.  Every wait of the model carries the absolute phase
it means; copies and MMAs complete at random later times, in order for each
issuing warp.  The model fails if a parity wait would answer differently from
the true one, or if the roles deadlock."""
import random

import pytest

WARPS = 2   # of a stream: enough for one to run ahead of another


class _Bar:
    def __init__(self, count):
        self.count, self.pending, self.phases = count, 0, 0

    def arrive(self):
        self.pending += 1
        assert self.pending <= self.count
        if self.pending == self.count:
            self.pending, self.phases = 0, self.phases + 1


def _simulate(tiles, seed, ring=8, acc_empty=True):
    """tiles: tiles of each item.  acc_empty: the products of an item wait until
    all elementwise warps have read the last item's sums."""
    rnd = random.Random(seed)
    bars, queues = {}, {"s": [], "d": [], "acc": [], "copies": []}
    for s in range(ring):
        bars["t_full", s], bars["t_empty", s] = _Bar(1), _Bar(1)
    for s in range(4):
        bars["s_full", s], bars["s_empty", s], bars["p_full", s] = _Bar(1), _Bar(1), _Bar(WARPS)
    for s in range(2):
        bars["own_full", s], bars["own_empty", s] = _Bar(1), _Bar(2)
        bars["d_full", s], bars["d_empty", s] = _Bar(1), _Bar(WARPS)
    bars["acc_full", 0], bars["acc_empty", 0] = _Bar(1), _Bar(2 * WARPS)

    def wait(name, i, phase):
        b = bars[name, i]
        while True:
            assert (b.phases & 1 != phase & 1) == (b.phases > phase), f"parity wait on {name}{i}"
            if b.phases > phase:
                return
            yield

    def producer():
        t = 0
        for n, count in enumerate(tiles):
            if n >= 2:
                yield from wait("own_empty", n & 1, (n >> 1) - 1)
            queues["copies"].append(("own_full", n & 1))
            for _ in range(count):
                if t >= ring:
                    yield from wait("t_empty", t % ring, t // ring - 1)
                queues["copies"].append(("t_full", t % ring))
                t += 1
                yield

    def scores(name, depth):
        t = 0
        for n, count in enumerate(tiles):
            yield from wait("own_full", n & 1, n >> 1)
            for j in range(count):
                yield from wait("t_full", t % ring, t // ring)
                if t >= depth:
                    yield from wait(name + "_empty", t % depth, t // depth - 1)
                queues[name].append((name + "_full", t % depth))
                if j + 1 == count:
                    queues[name].append(("own_empty", n & 1))
                t += 1
                yield

    def products():
        t = 0
        for n, count in enumerate(tiles):
            if n > 0 and acc_empty:
                yield from wait("acc_empty", 0, n - 1)
            for j in range(count):
                yield from wait("p_full", t & 3, t >> 2)
                queues["acc"] += [("s_empty", t & 3), ("t_empty", t % ring)]
                if j + 1 == count:
                    queues["acc"].append(("acc_full", 0))
                t += 1
                yield

    def elementwise(stream):
        t0 = 0
        for n, count in enumerate(tiles):
            for j in range((t0 ^ stream) & 1, count, 2):
                t = t0 + j
                yield from wait("s_full", t & 3, t >> 2)
                yield
                yield from wait("d_full", stream, t >> 1)
                yield
                bars["d_empty", stream].arrive()
                yield
                bars["p_full", t & 3].arrive()
            t0 += count
            yield from wait("acc_full", 0, n)
            yield
            bars["acc_empty", 0].arrive()

    roles = [producer(), scores("s", 4), scores("d", 2), products(),
             *(elementwise(i & 1) for i in range(2 * WARPS))]
    speed = [rnd.random() ** 2 + 0.05 for _ in roles]
    alive, quiet, state = list(range(len(roles))), 0, None
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


@pytest.mark.parametrize("most", [1, 2, 5, 20])
def test_barrier_phases(most):
    rng = random.Random(most)
    for trial in range(80):
        _simulate([rng.randint(1, most) for _ in range(rng.randint(1, 14))], trial)


def test_model_catches_sums_overwritten_early():
    """Without the wait for the last item's sums to be read, one stream's tile
    may run an item ahead of the other stream's warps: flagged."""
    flagged = 0
    for seed in range(60):
        tiles = [random.Random(seed).randint(1, 3) for _ in range(12)]
        _simulate(tiles, seed)
        try:
            _simulate(tiles, seed, acc_empty=False)
        except AssertionError:
            flagged += 1
    assert flagged > 0
