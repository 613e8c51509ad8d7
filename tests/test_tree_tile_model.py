"""attn_tree_tile.cu's roles, as a model on the CPU whose numbers are the kernel's: what each of them is for, and what happens when a wait gives up.

Waits: random interleavings of scout, converting warps, products and softmax warps.  With the kernel's own barriers every seed ends; with one barrier
for both products' ends, with a description written again one group earlier, and with a slot handed back by nobody, the model sees the fault.
Meetings: the four warps of a row meet on a named barrier, which has no limit; whichever wait gives up in any of them, all have to come to as
many meetings.
"""
import itertools
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_kv_cache_kvq_gb300", "csrc")
TILE = open(os.path.join(SRC, "attn_tree_tile.cu")).read()
VERIFY = open(os.path.join(SRC, "verify_runs.cu")).read()


def constant(name):
    return int(re.search(rf"constexpr int [^;]*\b{name} = (\d+)", TILE)[1])


SLOTS, GROUP, GROUPS = constant("kSlots"), constant("kGroup"), constant("kGroups")
PV_BARRIERS = int(re.search(r"uint64_t s_full\[2\], p_full\[2\], pv_done\[(\d)\];", TILE)[1])
LAG = GROUPS - 1
CONVERT, SOFTMAX = 3, 4  # warps of the model


class Fault(Exception):
    """What the model is there to see."""


def need(ok, what):
    if not ok:
        raise Fault(what)


class Bar:
    def __init__(self, count):
        self.count, self.n, self.phase = count, 0, 0

    def arrive(self):
        self.n += 1
        if self.n == self.count:
            self.n, self.phase = 0, self.phase + 1

    def over(self, k):
        """The parity test for phase k, which tells it from the one before alone."""
        need(k <= self.phase <= k + 1, f"a wait for phase {k} in phase {self.phase}")
        return self.phase == k + 1


def run(seed, pieces, pv_barriers=PV_BARRIERS, lag=LAG, empty_arrives=True):
    rnd = random.Random(seed)
    total, descs = sum(pieces), GROUP * GROUPS
    first = [i == 0 for p in pieces for i in range(p)]
    last = [i == p - 1 for p in pieces for i in range(p)]
    full, empty = [Bar(CONVERT) for _ in range(SLOTS)], [Bar(1) for _ in range(SLOTS)]
    s_full, p_full = [Bar(1), Bar(1)], [Bar(SOFTMAX), Bar(SOFTMAX)]
    pv_done = [Bar(1) for _ in range(pv_barriers)]
    q_full = Bar(SOFTMAX)
    desc_full, desc_done = [Bar(1) for _ in range(GROUPS)], [Bar(CONVERT) for _ in range(GROUPS)]
    queue, done = [], dict(S=-1, PV=-1)
    slot_of, desc = [None] * SLOTS, [None] * descs
    softmax_at, convert_at = [0] * SOFTMAX, [0] * CONVERT  # tiles that each warp is through with

    def wait(bar, k):
        while not bar.over(k):
            yield

    def wait_pv(tile):
        yield from wait(pv_done[tile % pv_barriers], tile // pv_barriers)
        need(done["PV"] == tile, "O of another tile")

    def scout():
        for g in range(-(-total // GROUP)):
            if g >= lag:
                v = g - lag
                yield from wait(desc_done[v % GROUPS], v // GROUPS)
            for tile in range(g * GROUP, min(total, g * GROUP + GROUP)):
                old = desc[tile % descs]
                need(old is None or min(softmax_at) > old and min(convert_at) > old and done["S"] >= old, "a description that is still read")
                desc[tile % descs] = tile
            yield
            desc_full[g % GROUPS].arrive()

    def convert(w):
        yield from wait(desc_full[0], 0)
        for tile in range(total):
            need(desc[tile % descs] == tile, "the description")
            ahead = min(tile + 1, total - 1)
            if ahead > tile and ahead % GROUP == 0:
                yield from wait(desc_full[ahead // GROUP % GROUPS], ahead // descs)
            need(desc[ahead % descs] == ahead, "the next description")
            for i in (2 * tile, 2 * tile + 1):
                if i >= SLOTS:
                    yield from wait(empty[i % SLOTS], i // SLOTS - 1)
                    need(done["PV" if i % 2 else "S"] >= (i - SLOTS) // 2, "a slot that is still read")
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
            need(slot_of[i % SLOTS] == i and desc[tile % descs] == tile, "K")
            if first[tile]:
                yield from wait(q_full, units)
                units += 1
            queue.append(("S", tile, i % SLOTS))

        yield from score(0)
        for tile in range(total):
            more = tile + 1 < total
            if more and not last[tile]:
                yield from score(tile + 1)
            yield from wait(p_full[tile & 1], tile >> 1)
            need(min(softmax_at) > tile, "weights")
            i = 2 * tile + 1
            yield from wait(full[i % SLOTS], i // SLOTS)
            need(slot_of[i % SLOTS] == i, "V")
            queue.append(("PV", tile, i % SLOTS))
            if more and last[tile]:
                yield from score(tile + 1)

    def tensor():
        while True:
            if queue:
                kind, tile, slot = queue.pop(0)
                yield
                done[kind] = tile
                (s_full[tile & 1] if kind == "S" else pv_done[tile % pv_barriers]).arrive()
                if empty_arrives:
                    empty[slot].arrive()
            else:
                yield

    def softmax(w):
        q_full.arrive()
        for tile in range(total):
            yield from wait(s_full[tile & 1], tile >> 1)
            need(done["S"] >= tile and desc[tile % descs] == tile, "S")
            if not first[tile] and rnd.random() < 0.3:  # O is rescaled
                yield from wait_pv(tile - 1)
            yield
            need(desc[tile % descs] == tile, "scales")
            softmax_at[w] = tile + 1
            p_full[tile & 1].arrive()
            if last[tile]:
                if tile + 1 < total:
                    yield
                    q_full.arrive()
                yield from wait_pv(tile)

    roles = [tensor(), products(), scout()] + [convert(w) for w in range(CONVERT)] + [softmax(w) for w in range(SOFTMAX)]
    live, pace = set(range(1, len(roles))), [1.0] * len(roles)
    for step in range(100000):
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
    raise Fault("stuck")


def work(seed):
    r = random.Random(1000 + seed)
    return [r.choice([1, 2, 3, r.randint(1, 40)]) for _ in range(r.randint(1, 5))]


def faults(**kw):
    """Whether one of 40 seeds sees a fault."""
    for seed in range(40):
        try:
            run(seed, work(seed), **kw)
        except Fault:
            return True
    return False


def test_the_kernels_barriers_serve():
    assert not faults()


@pytest.mark.parametrize("kw", [dict(pv_barriers=1), dict(lag=LAG + 1), dict(empty_arrives=False)])
def test_the_model_sees_what_each_of_them_is_for(kw):
    assert faults(**kw)


def test_the_waits_are_those_of_the_model():
    """The lag, and the barriers of tiles in turn, as the kernel has them."""
    assert "g >= kGroups - 1 && !wait_warp(&t->desc_done[(g - (kGroups - 1)) % kGroups], ((g - (kGroups - 1)) / kGroups) & 1u" in TILE
    assert "wait_for(&t->pv_done[buf ^ 1], ((jj - 1) >> 1) & 1u)" in TILE and "wait_for(&t->pv_done[buf], (jj >> 1) & 1u)" in TILE
    assert "commit(&t->pv_done[tile & 1], leader)" in TILE


# ------------------------------------------------------------------------------------------------ waits that give up
def walk(pieces, moves):
    """Waits and meetings of a warp over pieces of so many tiles (0: of a unit in which these 32 rows have none, which is one tile);
    ``moves``: tiles of the range where a maximum is outgrown and O is waited for."""
    tile = 0
    if pieces[0]:
        yield from ("meet", "meet")  # begin_unit
    for at, tiles in enumerate(pieces):
        for j in range(max(tiles, 1)):
            yield "wait"  # S
            if tiles:
                yield "meet"  # the vote
                if j and tile in moves:
                    yield "wait"  # O
            tile += 1
        if tiles:
            yield from ("meet", "meet")  # the row's sum
        if at + 1 < len(pieces) and pieces[at + 1]:
            yield from ("meet", "meet")  # begin_unit of the next
        yield "wait"  # O


def meetings(events, gives_up, leaves):
    n = waits = 0
    for e in events:
        if e == "meet":
            n += 1
        elif leaves and waits == gives_up:
            return n
        else:
            waits += 1
    return n


@pytest.mark.parametrize("pieces,moves", [([1], ()), ([3], (1,)), ([3, 1, 2], (1, 5)), ([2, 0, 0, 4], (3,)), ([0, 1], ()), ([5, 5], (1, 2, 3, 4, 6, 9))])
def test_warps_that_go_on_come_to_every_meeting(pieces, moves):
    events = list(walk(pieces, moves))
    where = [None, *range(events.count("wait"))]
    parts = [(i, j) for i, j in itertools.product(where, where)]
    assert all(meetings(events, i, False) == meetings(events, j, False) for i, j in parts)
    assert any(meetings(events, i, True) != meetings(events, j, True) for i, j in parts)  # the model sees warps that are left alone


def body(src, head, end="\n}\n"):
    role = src[src.index(head):]
    return re.sub(r"//[^\n]*", "", role[:role.index(end)])


def test_the_softmax_role_has_no_way_out_but_its_end():
    role = body(TILE, "__device__ void softmax_role(")
    assert role.count("return") == 1 and "return r != 0;" in role  # of the vote
    # every meeting is under conditions that the four warps of a row share: none looks at whether a wait gave up
    for line in re.findall(r"[^\n]*meet(?:_any)?\([^\n]*", role):
        assert "alive" not in line
    for block in re.findall(r"if \(([^{};]*)\) \{\n[^{}]*\bmeet\(\)", role):
        assert block.strip() in ("active", "had"), block


def test_tensor_memory_is_given_back_behind_the_last_product():
    kernel = TILE[TILE.index("tree_tile_kernel(const __grid_constant__"):]
    order = [kernel.index(x) for x in ("mma_role(", "commit(&t->drained", "mbar_try_wait(&t->drained", "__syncthreads();\n  fence_after();\n  if (warp == kMmaWarp)",
                                       "tcgen05.dealloc")]
    assert order == sorted(order) and "drained" not in body(TILE, "__device__ void mma_role(")
    assert kernel[kernel.index("softmax_role("):kernel.index("tcgen05.dealloc")].count("return") == 0


def test_a_walk_whose_exchange_gives_up_ends_with_its_cluster():
    """verify_runs.cu: behind the tree's hand-over no block leaves before the last cluster barrier, and no loop goes on without its exchange."""
    kernel = body(VERIFY, "verify_kernel(const VerifyArgs a) {")
    walk_of = kernel[kernel.index("int cur = 0, kept = 1"):]
    assert "return" not in walk_of and walk_of.rstrip().endswith("cluster.sync();")
    loops = re.findall(r"(?:for|while) \(([^{}]*)\) \{", walk_of)
    assert [x for x in loops if "step < n" in x][0].endswith("++step") and "step < n && alive" in walk_of
    assert "while (child < n && alive)" in walk_of and walk_of.index("if (!alive) break;") < walk_of.index("last = drawn;")
    exchange = kernel[kernel.index("auto exchange ="):kernel.index("auto total =")]
    assert "while (alive && !try_wait_cluster(" in exchange and "kWaitClocks" in exchange
    assert exchange.count("return") == 1  # of the pair that is sent
