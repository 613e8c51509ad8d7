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


# ------------------------------------------------------------------------------------------------ shared pages
SHARED = dict(new=[-1, 0, 20], lens=[20, 25, 0], stack=[3, -9, -9, -9], count=1, rows=20,
              table=[[5, 1, -1], [5, 2, -1], [-1, -1, -1]])  # requests 0 and 1 have page 5, a common prefix; 0 is finished


def test_oracle_keeps_a_shared_page():
    s = SHARED
    args = (s["new"], s["lens"], s["stack"], s["count"], np.array(s["table"], dtype=np.int32), s["rows"])
    m = R.map_runs(*args, kept=[1, 0, 0])
    assert m["ok"] and m["table"][2].tolist() == [1, 3, -1] and m["count"] == 0  # not page 5
    assert not R.map_runs(*args, kept=[3, 0, 0])["ok"] and not R.map_runs(*args, kept=[-1, 0, 0])["ok"]
    m = R.map_runs([-1, -1, 0], *args[1:], kept=[1, 0, 7])  # then the last that has it
    assert m["stack"].tolist() == [3, 1, 5, 2]


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to("cuda", dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3p", "int8p"])
def test_a_prefix_outlives_the_first_request_that_had_it(kvq, fmt):  # noqa: F811
    """Requests 0 and 1 share their first page; 0 ends, 2 starts and writes its pages: request 1 still reads its prefix."""
    H, Hq, pages = 2, 4, 6
    cache = kvq.PagedCache(fmt, fmt, H, pages)
    table = dev(np.array(SHARED["table"]))
    x = torch.randn(45, 2 * H, 128, device="cuda").bfloat16()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # the prefix with request 0's own tokens, then request 1's own tokens behind the same prefix
    kvq.append_runs(cache, x[:20, :H], x[:20, H:], dev([20, 0, 0]), table, run_starts=dev([0, 20, 20, 20]), err=err)
    kvq.append_runs(cache, x[20:29, :H], x[20:29, H:], dev([0, 25, 0]), table, run_starts=dev([0, 0, 9, 9]), err=err)
    q = torch.randn(3, Hq, 128, device="cuda").bfloat16()
    ws = torch.empty(kvq.attn_runs_workspace_size(3, 3, 1, H, Hq, q.dtype), dtype=torch.uint8, device="cuda")

    def attend(lens):
        out = torch.empty_like(q)
        kvq.attn_runs(cache, q, dev(lens), table, out, ws, err=err)
        return out[1].clone()

    before = attend([20, 25, 0])
    new, lens, stack, count = dev(SHARED["new"]), dev(SHARED["lens"]), dev(SHARED["stack"]), dev([SHARED["count"]])
    starts = dev([0] * 4)
    kvq.map_runs(new, lens, stack, count, table, starts, lens, count, kept_pages=dev([1, 0, 0]), err=err)
    assert table[2, :2].tolist() == [1, 3] and count.item() == 0 and lens.tolist() == [0, 25, 20]
    kvq.append_runs(cache, x[25:, :H], x[25:, H:], lens, table, run_starts=starts, err=err)
    assert torch.equal(attend([0, 25, 20]), before)
    assert err.item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [7, 400])
def test_kept_pages_equal_the_oracle(kvq, batch):  # noqa: F811
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 200, batch)
    new = np.where(rng.random(batch) < 0.4, -1, rng.integers(0, 40, batch))
    kept = np.array([rng.integers(0, -(-n // 16) + 1) for n in lens])
    table, total = tables(rng, lens, width=16)
    stack = np.full(2 * total, -9)
    stack[:total] = total + np.arange(total)
    for bad in (None, -1, 1):
        k = kept.copy()
        k[new >= 0] = 99  # not looked at
        if bad is not None:
            s = np.flatnonzero(new < 0)[-1]
            k[s] = -1 if bad < 0 else -(-lens[s] // 16) + 1
        ref = R.map_runs(new, lens, stack, total, table, int(np.maximum(new, 0).sum()), kept=k)
        assert ref["ok"] == (bad is None)
        t = dict(new=dev(new), lens=dev(lens), stack=dev(stack), count=dev([total]), table=dev(table))
        starts, err = dev(np.full(batch + 1, -7)), torch.zeros(1, dtype=torch.int32, device="cuda")
        kvq.map_runs(t["new"], t["lens"], t["stack"], t["count"], t["table"], starts, t["lens"], t["count"], kept_pages=dev(k), err=err)
        assert err.item() == (0 if ref["ok"] else 5)
        assert np.array_equal(t["stack"].cpu().numpy(), ref["stack"]) and np.array_equal(t["table"].cpu().numpy(), ref["table"])
        assert t["lens"].tolist() == list(ref["seq_lens"]) and t["count"].item() == ref["count"] and starts.tolist() == ref["run_starts"].tolist()


# ------------------------------------------------------------------------------------------------ pages behind a length set back
def drafts(step, batch=5):
    """Steps of drafts: each request adds some tokens, then all but a few of them are rejected; sometimes one is finished."""
    rng = np.random.default_rng(100 * batch + step)
    new = rng.integers(0, 40, batch)
    if step % 4 == 3:
        new[rng.integers(batch)] = -1
    return new, rng.random(batch)


def test_oracle_loses_no_page_to_rejected_drafts():
    B, width, pages = 5, 12, 80
    lens, table, stack, count, held = np.zeros(B, int), np.full((B, width), -1), np.arange(pages), pages, np.zeros(B, int)
    for step in range(60):
        new, share = drafts(step)
        new = np.where(lens + new > width * 16, -1, new)
        m = R.map_runs(new, lens, stack, count, table, 200, held=held)
        assert m["ok"]
        lens, table, stack, count, held = m["seq_lens"], m["table"], m["stack"], m["count"], m["held"]
        owned = [int(p) for s in range(B) for p in table[s, :held[s]]] + stack[:count].tolist()
        assert sorted(owned) == list(range(pages))  # every page has one owner
        lens = np.where(new > 0, lens - (share * np.maximum(new, 0)).astype(int), lens)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,in_graph", [(5, True), (300, False)])
def test_rejected_drafts_keep_their_pages(kvq, batch, in_graph):  # noqa: F811
    """Captured once and replayed in place, the lengths set back between the steps; every step against the oracle."""
    width, pages, rows = 12, 16 * batch, 40 * batch
    lens, table, stack, count, held = np.zeros(batch, int), np.full((batch, width), -1), np.arange(pages), pages, np.zeros(batch, int)
    t = dict(new=dev(np.zeros(batch)), lens=dev(lens), stack=dev(stack), count=dev([count]), table=dev(table), held=dev(held),
             starts=dev(np.zeros(batch + 1)), slots=dev(np.zeros(rows)), pos=dev(np.zeros(rows)))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        kvq.map_runs(t["new"], t["lens"], t["stack"], t["count"], t["table"], t["starts"], t["lens"], t["count"], slot_mapping=t["slots"],
                     positions=t["pos"], held_pages=t["held"], err=err)

    call()  # no tokens: nothing changes
    torch.cuda.synchronize()
    run = call
    if in_graph:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        run = graph.replay
    for step in range(12):
        new, share = drafts(step, batch)
        new = np.where(lens + new > width * 16, -1, new)
        t["new"].copy_(dev(new))
        run()
        m = R.map_runs(new, lens, stack, count, table, rows, held=held)
        assert m["ok"] and err.item() == 0
        lens, table, stack, count, held = m["seq_lens"], m["table"], m["stack"], m["count"], m["held"]
        got = {k: v.cpu().numpy() for k, v in t.items()}
        for a, b in (("lens", lens), ("table", table), ("stack", stack), ("held", held), ("starts", m["run_starts"]), ("slots", m["slots"]),
                     ("pos", m["positions"])):
            assert np.array_equal(got[a], b), (step, a)
        assert got["count"][0] == count
        lens = np.where(new > 0, lens - (share * np.maximum(new, 0)).astype(int), lens)
        t["lens"].copy_(dev(lens))


@pytest.mark.gpu
@pytest.mark.parametrize("held", [[1, 2, 0], [2, 2, -1], [2, 4, 0]])
def test_a_wrong_number_of_held_pages_is_refused(kvq, held):  # noqa: F811
    table = np.array(SHARED["table"], dtype=np.int32)
    lens, stack = SHARED["lens"], SHARED["stack"]
    assert not R.map_runs([0, 1, 0], lens, stack, 1, table, 9, held=held)["ok"]
    t = [dev([0, 1, 0]), dev(lens), dev(stack), dev([1]), dev(table), dev([7] * 4)]
    h, err = dev(held), torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.map_runs(*t, t[1], t[3], held_pages=h, err=err)
    assert err.item() == 5 and h.tolist() == held and t[1].tolist() == lens and t[2].tolist() == stack and t[3].tolist() == [1]
    assert t[4].tolist() == table.tolist() and t[5].tolist() == [0] * 4
    # kept and held together: all that a finished request has, but the shared page
    h, err, pages = dev([3, 2, 0]), torch.zeros_like(err), dev([[5, 1, 0], [5, 2, -1], [-1, -1, -1]])
    kvq.map_runs(dev([-1, 1, 0]), *t[1:4], pages, t[5], t[1], t[3], kept_pages=dev([1, 0, 0]), held_pages=h, err=err)
    assert err.item() == 0 and t[2].tolist() == [3, 1, 0, -9] and t[3].tolist() == [3] and h.tolist() == [0, 2, 0]
