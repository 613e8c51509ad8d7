"""The waits of attn_tree_tile.cu's roles, as a model on the CPU: random interleavings of converting warps, products, softmax warps and scout.

A wait on an mbarrier tells a phase from the one before it by its parity alone.  For every wait the model asserts that no other
phase can be the current one (else a wait would pass too early, or never), that what the wait is for has happened when it passes, that no
slot or description is written while it is still read, and that all roles end.
"""
import random

import pytest

SLOTS, BUFS, GROUP, GROUPS = 6, 5, 4, 4
CONVERT, TEAMS, QUARTERS = 3, 4, 2  # warps of the model: a warp of each team for each quarter of the rows


class Meeting:
    """A named barrier of the warps that have the same rows."""

    def __init__(self):
        self.n = self.round = 0

    def meet(self):
        mine = self.round
        self.n += 1
        if self.n == TEAMS:
            self.n, self.round = 0, mine + 1
        while self.round == mine:
            yield


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
    """Half tile u has keys 64 (u & 1) .. of tile u >> 1; a piece is some tiles of one unit."""
    rnd = random.Random(seed)
    total = sum(pieces)
    starts = [sum(pieces[:n]) for n in range(len(pieces))]
    piece_of = [n for n, p in enumerate(pieces) for _ in range(p)]
    rows = [[True] + [rnd.random() < 0.6 for _ in range(QUARTERS - 1)] for _ in pieces]  # quarters that the piece's unit has rows in
    full, empty = [Bar(CONVERT) for _ in range(SLOTS)], [Bar(1) for _ in range(SLOTS)]
    s_full, p_full, pv_done = ([Bar(n) for _ in range(BUFS)] for n in (1, QUARTERS, 1))
    m_ready = [[Bar(1) for _ in range(QUARTERS)] for _ in range(TEAMS)]
    q_full = Bar(TEAMS * QUARTERS)
    desc_full, desc_done = [Bar(1) for _ in range(GROUPS)], [Bar(CONVERT) for _ in range(GROUPS)]
    meetings = [Meeting() for _ in range(QUARTERS)]
    queues = {"S": [], "PV": []}
    done = {"S": -1, "PV": -1}  # half tiles
    slot_of, desc = [None] * SLOTS, [None] * (GROUP * GROUPS)
    weighed = [[-1] * QUARTERS for _ in range(2 * total)]  # half tiles whose weights are there
    maximum = [-1] * QUARTERS  # the half tile that the running maximum is of
    staged = [0] * len(pieces)  # warps that have put the piece's query there
    read = [0] * len(pieces)  # warps that have read the piece's O
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
                assert old is None or (done["PV"] >= 2 * old + 1 and min(convert_at) > old)
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
                    assert done["PV" if (i - SLOTS) % 2 else "S"] >= (i - SLOTS) // 2 * 2 + 1
                slot_of[i % SLOTS] = i
                yield
                full[i % SLOTS].arrive()
            convert_at[w] = tile + 1
            if tile % GROUP == GROUP - 1 or tile + 1 == total:
                desc_done[tile // GROUP % GROUPS].arrive()
        for i in range(max(0, 2 * total - SLOTS), 2 * total):
            yield from wait(empty[i % SLOTS], i // SLOTS)

    def score():
        for u in range(2 * total):
            tile, i = u >> 1, u >> 1 << 1
            if u & 1 == 0:
                yield from wait(full[i % SLOTS], i // SLOTS)
                assert desc[tile % (GROUP * GROUPS)] == tile
                if tile in starts:
                    p = starts.index(tile)
                    yield from wait(q_full, p)
                    assert staged[p] == TEAMS * QUARTERS
            if u >= BUFS:
                yield from wait(pv_done[u % BUFS], u // BUFS - 1)
                assert done["PV"] >= u - BUFS
            assert slot_of[i % SLOTS] == i
            queues["S"].append((u, i % SLOTS if u & 1 else None))

    def pv():
        for u in range(2 * total):
            i = (u >> 1) * 2 + 1
            if u & 1 == 0:
                yield from wait(full[i % SLOTS], i // SLOTS)
                assert slot_of[i % SLOTS] == i and desc[(u >> 1) % (GROUP * GROUPS)] == u >> 1
            yield from wait(p_full[u % BUFS], u // BUFS)
            assert weighed[u] == [u] * QUARTERS
            p = piece_of[u >> 1]
            if p and u == 2 * starts[p]:  # writes over the O of the piece before
                assert read[p - 1] == TEAMS * sum(rows[p - 1])
            queues["PV"].append((u, i % SLOTS if u & 1 else None))

    def tensor(kind):
        while True:
            if queues[kind]:
                u, slot = queues[kind].pop(0)
                yield
                assert done[kind] == u - 1
                done[kind] = u
                (s_full if kind == "S" else pv_done)[u % BUFS].arrive()
                if slot is not None:
                    empty[slot].arrive()
            else:
                yield

    def softmax(team, quarter):
        def stage(p):
            if rows[p][quarter]:
                for _ in range(2):
                    yield from meetings[quarter].meet()
            staged[p] += 1
            q_full.arrive()

        yield from stage(0)
        for p, size in enumerate(pieces):
            had = rows[p][quarter]
            for tile in range(starts[p], starts[p] + size):
                if tile & 1 != team >> 1:
                    continue
                u = 2 * tile + (team & 1)
                yield from wait(s_full[u % BUFS], u // BUFS)
                assert done["S"] >= u and desc[tile % (GROUP * GROUPS)] == tile
                if u:
                    yield from wait(m_ready[(u - 1) & 3][quarter], (u - 1) >> 2)
                assert maximum[quarter] == u - 1
                yield
                maximum[quarter] = u
                m_ready[team][quarter].arrive()
                if had and u != 2 * starts[p] and rnd.random() < 0.3:  # O is rescaled
                    yield from wait(pv_done[(u - 1) % BUFS], (u - 1) // BUFS)
                    assert done["PV"] == u - 1
                yield
                weighed[u][quarter] = u
                p_full[u % BUFS].arrive()
            if had:
                yield from meetings[quarter].meet()
            e = 2 * (starts[p] + size) - 1
            yield from wait(s_full[e % BUFS], e // BUFS)
            assert done["S"] == e  # nothing reads the query that is written over
            if p + 1 < len(pieces):
                yield from stage(p + 1)
            if had:
                yield from wait(pv_done[e % BUFS], e // BUFS)
                assert done["PV"] == e
                yield
                read[p] += 1
                yield from meetings[quarter].meet()

    roles = [tensor("S"), tensor("PV"), score(), pv(), scout()] + [convert(w) for w in range(CONVERT)]
    roles += [softmax(t, q) for t in range(TEAMS) for q in range(QUARTERS)]
    live = set(range(2, len(roles)))
    pace = [1.0] * len(roles)
    for step in range(400000):
        if not live:
            return
        if step % 300 == 0:  # who is slow changes all the time
            pace = [rnd.random() ** 4 + 0.005 for _ in roles]
        i = rnd.choices(range(len(roles)), pace)[0]
        if i > 1 and i not in live:
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


def test_one_barrier_for_all_products_would_not_do():
    """The model sees the fault that a barrier for each buffer mends: with one for all P V, a warp at a piece's end may find it phases behind."""
    bar = Bar(1)
    bar.arrive()  # P V of half tile 0 is over, that of 1 is running, a warp is at the end of half tile 2
    with pytest.raises(AssertionError):
        bar.over(2)
