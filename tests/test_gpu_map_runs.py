"""kvq_map_runs: steps that cannot be taken, shared pages, pages held beyond a length (GPU; the oracle's pins are below, on the CPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import runs as R  # noqa: E402
from tests.runs_cases import tables  # noqa: E402
from tests.test_gpu_runs import check_map, kvq, run_map  # noqa: E402,F401

ODD = [-1, -(1 << 31), R.MAX_PAGE + 1, (1 << 31) - 1]


def odd_step(where, odd, batch):
    """A step of ``batch`` requests, some finished, one page number of which cannot be: (new, lens, stack, count, table, rows)."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(17, 100, batch)
    lens[lens % 16 == 0] += 1
    gone = np.arange(batch) % 8 == 1
    new = np.where(gone, -1, 0 if where == "pushed" else rng.integers(30, 60, batch))  # pushed: more comes back than goes out
    new[[0, 2]] = 0 if where == "pushed" else 40, 0
    table, total = tables(rng, lens, width=12)
    want = int(sum(max(0, -(-(l + n) // 16) - -(-l // 16)) for l, n in zip(lens, new) if n > 0))
    back = int(sum(-(-l // 16) for l, n in zip(lens, new) if n < 0))
    count = want + 3
    stack = np.full(count + back, -9)
    stack[:count] = total + np.arange(count)
    gone = np.flatnonzero(gone)
    if where == "popped":
        assert want > back
        stack[count - 1] = odd
    elif where in ("handed on", "pushed"):  # the last page that comes back: the first to go out, or one that stays on the stack
        s = gone[-1]
        table[s, -(-lens[s] // 16) - 1] = odd
    elif where == "gone on in":
        table[0, lens[0] // 16] = odd
    else:  # entries that the step does not touch
        stack[0] = odd
        table[2, lens[2] // 16] = odd
        table[0, lens[0] // 16 - 1] = odd
        table[gone[0], -(-lens[gone[0]] // 16)] = odd
    return new, lens, stack, count, table, int(np.maximum(new, 0).sum()) + 5


WHERE = ["popped", "handed on", "pushed", "gone on in", "elsewhere"]


@pytest.mark.parametrize("where", WHERE)
def test_oracle_refuses_a_step_with_a_page_that_cannot_be(where):
    for odd in ODD:
        assert R.map_runs(*odd_step(where, odd, 9))["ok"] == (where == "elsewhere")
    assert R.map_runs(*odd_step(where, R.MAX_PAGE, 9))["ok"]


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch", [9, 200])  # one block, eight
@pytest.mark.parametrize("where", WHERE)
def test_a_page_that_cannot_be_stops_the_whole_step(kvq, where, batch, in_place):  # noqa: F811
    for odd in ODD:
        step = odd_step(where, odd, batch)
        ref = R.map_runs(*step)
        assert ref["ok"] == (where == "elsewhere")
        got, err = run_map(kvq, *step, in_place)
        assert err == (0 if ref["ok"] else 5)
        check_map(got, ref)
