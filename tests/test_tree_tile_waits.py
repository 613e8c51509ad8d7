"""The waits of attn_tree_tile.cu's roles, as a model on the CPU: random interleavings of converting warps, products, softmax warps and scout.

A wait on an mbarrier tells a phase from the one before it by its parity alone.  For every wait the model asserts that no other
phase can be the current one (else a wait would pass too early, or never), that what the wait is for has happened when it passes, that no
slot or description is written while it is still read, and that all roles end.
"""
import random

import pytest

SLOTS, GROUP, GROUPS = 6, 4, 4
CONVERT, SOFTMAX = 3, 4  # warps of the model


class Bar:
    def __init__(self, count):
        self.count, self.n, self.phase = count, 0, 0

    def arrive(self):
        self.n += 1
        if self.n == self.count:
            self.n, self.phase = 0, self.phase + 1

    def over(self, k):
        """The parity test for phase k."""
        assert k <= self.phase <= k + 1, (k, self.phase)
        return (self.phase & 1) != (k & 1)


def run(seed, pieces):
    rnd = random.Random(seed)
    total = sum(pieces)
    first = [i == 0 for p in pieces for i in range(p)]
    last = [i == p - 1 for p in pieces for i in range(p)]
    full, empty = [Bar(CONVERT) for _ in range(SLOTS)], [Bar(1) for _ in range(SLOTS)]
    s_full, p_full, pv_done = ([Bar(n), Bar(n)] for n in (1, SOFTMAX, 1))
    q_full = Bar(SOFTMAX)
    desc_full, desc_done = [Bar(1) for _ in range(GROUPS)], [Bar(CONVERT) for _ in range(GROUPS)]
    tensor_queue = []
    done = dict(S=-1, PV=-1)
    slot_of, desc = [None] * SLOTS, [None] * (GROUP * GROUPS)
    softmax_at = [0] * SOFTMAX  # tiles that each warp is through with
    convert_at = [0] * CONVERT

    def wait(bar, k):
        while not bar.over(k):
            yield

    def scout():
        for g in range(-(-total // GROUP)):
            if g >= GROUPS - 1:
                v = g - (GROUPS - 1)
                yield from wait(desc_done[v % GROUPS], v // GROUPS)
            for tile in range(g * GROUP, min(total, g * GROUP + GROUP)):
                old = desc[tile % (GROUP * GROUPS)]
                assert old is None or (min(softmax_at) > old and min(convert_at) > old and done["S"] >= old)
                desc[tile % (GROUP * GROUPS)] = tile
            yield
            desc_full[g % GROUPS].arrive()

    def convert(w):
        yield from wait(desc_full[0], 0)
        for tile in range(total):
            assert desc[tile % (GROUP * GROUPS)] == tile
            ahead = min(tile + 1, total - 1)
            if ahead > tile and ahead % GROUP == 0:
                yield from wait(desc_full[ahead // GROUP % GROUPS], ahead // (GROUP * GROUPS))
            assert desc[ahead % (GROUP * GROUPS)] == ahead
            for i in (2 * tile, 2 * tile + 1):
                if i >= SLOTS:
                    yield from wait(empty[i % SLOTS], i // SLOTS - 1)
                    assert done["PV" if i % 2 else "S"] >= (i - SLOTS) // 2
                slot_of[i % SLOTS] = i
                yield
                full[i % SLOTS].arrive()
            convert_at[w] = tile + 1
            if tile % GROUP == GROUP - 1 or tile + 1 == total:
                desc_done[tile // GROUP % GROUPS].arrive()
        for i in range(max(0, 2 * total - SLOTS), 2 * total):
            yield from wait(empty[i % SLOTS], i // SLOTS)

    def products():
        units = 0

        def score(tile):
            nonlocal units
            i = 2 * tile
            yield from wait(full[i % SLOTS], i // SLOTS)
            assert slot_of[i % SLOTS] == i and desc[tile % (GROUP * GROUPS)] == tile
            if first[tile]:
                yield from wait(q_full, units)
                units += 1
            tensor_queue.append(("S", tile, i % SLOTS))

        yield from score(0)
        for tile in range(total):
            more = tile + 1 < total
            if more and not last[tile]:
                yield from score(tile + 1)
            yield from wait(p_full[tile & 1], tile >> 1)
            assert min(softmax_at) > tile
            i = 2 * tile + 1
            yield from wait(full[i % SLOTS], i // SLOTS)
            assert slot_of[i % SLOTS] == i
            tensor_queue.append(("PV", tile, i % SLOTS))
            if more and last[tile]:
                yield from score(tile + 1)

    def tensor():
        while True:
            if tensor_queue:
                kind, tile, slot = tensor_queue.pop(0)
                yield
                assert done[kind] == tile - 1
                done[kind] = tile
                (s_full if kind == "S" else pv_done)[tile & 1].arrive()
                empty[slot].arrive()
            else:
                yield

    def softmax(w):
        q_full.arrive()
        for tile in range(total):
            yield from wait(s_full[tile & 1], tile >> 1)
            assert done["S"] >= tile and desc[tile % (GROUP * GROUPS)] == tile
            if not first[tile] and rnd.random() < 0.3:  # O is rescaled
                yield from wait(pv_done[(tile - 1) & 1], (tile - 1) >> 1)
                assert done["PV"] == tile - 1
            yield
            softmax_at[w] = tile + 1
            p_full[tile & 1].arrive()
            if last[tile]:
                if tile + 1 < total:
                    yield
                    q_full.arrive()
                yield from wait(pv_done[tile & 1], tile >> 1)
                assert done["PV"] == tile

    roles = [tensor(), products(), scout()] + [convert(w) for w in range(CONVERT)] + [softmax(w) for w in range(SOFTMAX)]
    live = set(range(1, len(roles)))
    pace = [1.0] * len(roles)
    for step in range(200000):
        if not live:
            return
        if step % 300 == 0:  # who is slow changes all the time
            pace = [rnd.random() ** 4 + 0.005 for _ in roles]
        i = rnd.choices(range(len(roles)), pace)[0]
        if i and i not in live:
            continue
        try:
            next(roles[i])
        except StopIteration:
            live.discard(i)
    raise AssertionError("stuck")


@pytest.mark.parametrize("seed", range(120))
def test_every_wait_ends_and_is_for_what_it_says(seed):
    r = random.Random(seed)
    run(seed, [r.choice([1, 2, 3, r.randint(1, 30)]) for _ in range(r.randint(1, 5))])


def test_one_barrier_for_both_products_would_not_do():
    """The model sees the fault that two barriers mend: with one barrier for all P V, a warp at a piece's end may find it a phase behind."""
    bar = Bar(1)
    bar.arrive()  # P V of tile 0 is over, that of tile 1 is running, a warp is at the end of tile 2
    with pytest.raises(AssertionError):
        bar.over(2)
