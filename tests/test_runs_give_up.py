"""The two warps of a row in the tile kernel of kvq_attn_runs, when a bounded wait gives up (CPU).

The pair meets on a named barrier, which has no limit: a meeting that one of them does not come to never ends.  ``walk`` is the
order of waits and meetings in ``softmax_role``; whichever wait gives up in either warp, both have to come to as many meetings.
"""
import itertools
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_kv_cache_kvq_gb300", "csrc", "attn_runs_tile.cu")


def walk(pieces, moves):
    """Waits and meetings of a warp over pieces of so many tiles (0: a piece whose rows are all in the other half); ``moves``: the
    tiles, counted over the range, where a maximum is outgrown and O is waited for."""
    tile, staged = 0, False
    for p, tiles in enumerate(pieces):
        for j in range(tiles):
            if not staged:
                yield from ("meet", "meet")  # begin_unit
                staged = True
            yield "wait"  # S
            yield "meet"  # the row's maximum
            if j and tile in moves:
                yield "wait"  # O
            tile += 1
        if tiles:
            yield from ("meet", "meet")  # the row's sum
            staged = False
            if p + 1 < len(pieces) and pieces[p + 1]:
                yield from ("meet", "meet")  # begin_unit of the next
                staged = True
            yield "wait"  # O


def meetings(events, gives_up, leaves):
    """Meetings that a warp comes to whose wait number ``gives_up`` fails (None: none does)."""
    n = waits = 0
    for e in events:
        if e == "meet":
            n += 1
        else:
            if waits == gives_up and leaves:
                return n + 1  # the peer released once
            waits += 1
    return n


CASES = [([1], ()), ([3], (1,)), ([3, 1, 2], (1, 5)), ([2, 0, 0, 4], (3,)), ([0, 1], ()), ([5, 5], (1, 2, 3, 4, 6, 9))]


def stuck(pieces, moves, leaves):
    events = list(walk(pieces, moves))
    where = [None, *range(events.count("wait"))]
    return [(i, j) for i, j in itertools.product(where, where) if meetings(events, i, leaves) != meetings(events, j, leaves)]


@pytest.mark.parametrize("pieces,moves", CASES)
def test_a_warp_that_goes_on_comes_to_every_meeting(pieces, moves):
    assert not stuck(pieces, moves, leaves=False)
    assert stuck(pieces, moves, leaves=True)  # the model sees a pair that is left alone


def test_the_role_has_no_way_out_but_its_end():
    src = open(SRC).read()
    role = src[src.index("__device__ void softmax_role("):]
    role = role[:role.index("\n}\n")]
    role = re.sub(r"auto exchange = .*?\n  };", "", role, flags=re.S)
    assert "wait_for(" in role and "return" not in re.sub(r"//[^\n]*", "", role)
    assert "bar.arrive" not in role


def test_tensor_memory_is_given_back_behind_the_last_product():
    """On every path: the issuing warp's last commit is waited for before the block frees TMEM and ends, by no length of time."""
    src = open(SRC).read()
    assert "__nanosleep" not in src
    kernel = src[src.index("tile_kernel(const __grid_constant__"):]
    order = [kernel.index(x) for x in ("mma_role(", "commit(&t->drained", "mbar_try_wait(&t->drained", "__syncthreads();\n  fence_after();\n  if (warp == kMmaWarp)",
                                       "tcgen05.dealloc")]
    assert order == sorted(order)
    role = src[src.index("__device__ void mma_role("):src.index("// ---", src.index("__device__ void mma_role("))]
    assert "drained" not in role  # its early returns do not pass it by
