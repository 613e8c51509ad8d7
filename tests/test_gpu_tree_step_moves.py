"""Speculative steps whose drafts are often accepted (GPU): tokens move, across pages and under other scales, and steps go on from there.

The vocabulary has four tokens, two whose values are small and two whose values are large, and all values double from step to step.  A tree's early
rows hold the small ones, its late rows the large ones, and a row with children of both kinds goes on, whatever is chosen: a late row is then kept in
a page whose tokens were all smaller.  Every test says how many tokens were accepted, moved, and made a page's scale grow at least.
"""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import tests.test_gpu_tree_step as step_of  # noqa: E402
from oracle import runs as R  # noqa: E402
from oracle import trees as T  # noqa: E402
from tests.runs_cases import starts_of, unpack  # noqa: E402
from tests.test_gpu_tree_step import G, H, Server  # noqa: E402
from tests.tree_cases import distribution  # noqa: E402

VOCAB, STEPS = 4, 20


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


@pytest.fixture(autouse=True)
def few_tokens(monkeypatch):
    monkeypatch.setattr(step_of, "V", VOCAB)


class Between:
    """The library with the verification given draft probabilities, and the cache looked at before tokens are kept."""

    def __init__(self, kvq, server):
        self.kvq, self.server = kvq, server

    def __getattr__(self, name):
        return getattr(self.kvq, name)

    def verify_runs(self, *a, **kw):
        if self.server.draft is not None:
            kw["draft"] = self.server.draft
        self.kvq.verify_runs(*a, **kw)

    def keep_runs(self, *a, **kw):
        if self.server.watch:
            self.server.before = [t.clone() for c in self.server.caches for t in (c.k, c.v, c.k_scale, c.v_scale)]
        self.kvq.keep_runs(*a, **kw)


def server_of(kvq, fmt, batch, n, seed, how="target", dtype=torch.bfloat16, watch=False):
    s = Server(kvq, fmt, batch, n, seed, dtype=dtype, greedy=how == "greedy")
    s.embed[:, :, H * G + H:] *= torch.tensor([1 / 16, 1 / 8, 1 / 2, 1.0], device="cuda").to(dtype)[None, :, None, None]
    s.draft = torch.zeros((s.rows, VOCAB), device="cuda") if how == "draft" else None
    s.watch, s.before, s.kvq = watch, None, Between(kvq, s)
    return s


def drafts(rng, batch, n, last):
    """Trees of n / 2 to n rows: early rows below any row before them, the first two of them below the root, with tokens 0 and 1 in turn; then late
    rows, the same with tokens 2 and 3."""
    trees, tokens = [], []
    for s in range(batch):
        size = int(rng.integers((n + 1) // 2, n + 1))
        late = (size + 1) // 2
        tree = [-1] + [0 if i in (1, 2, late, late + 1) else int(rng.integers(0, i)) for i in range(1, size)]
        trees.append(tree)
        tokens += [int(last[s])] + [i % 2 if i < late else 2 + i % 2 for i in range(1, size)]
    return trees, tokens


def feed(server, rng, last):
    trees, tokens = drafts(rng, server.B, server.n, last)
    if server.draft is not None:
        server.draft.copy_(torch.as_tensor(np.stack([distribution(rng, VOCAB, 0.5) for _ in range(server.rows)])))
    server.feed(trees, tokens, torch.as_tensor(rng.random((server.rows, 2)).astype(np.float32)))
    return trees, tokens


class Tally:
    accepted = moved = across = 0

    def add(self, starts, keep, kept, lens):
        """lens: with the kept tokens."""
        for s, m in enumerate(kept):
            path = keep[starts[s]:starts[s] + m]
            self.accepted += m - 1
            p0 = lens[s] - m
            self.moved += any(j != i for j, i in enumerate(path))
            self.across += any((p0 + i) // 16 != (p0 + j) // 16 for j, i in enumerate(path))


def run_steps(server, rng, count, run, tally=None):
    """Yields the accepted tokens of every request, step by step."""
    last = rng.integers(0, VOCAB, server.B)
    for _ in range(count):
        trees, tokens = feed(server, rng, last)
        run()
        torch.cuda.synchronize()
        assert server.err.item() == 0
        starts, kept, keep = starts_of([len(t) for t in trees]), server.kept.tolist(), server.keep.tolist()
        if tally:
            tally.add(starts, keep, kept, server.lens.tolist())
        last = np.array(server.next.tolist())
        server.embed[:, :, H * G + H:] *= 2  # the next step's values; what is chosen goes by the same scores
        server.head *= 0.5
        yield [[tokens[starts[s] + keep[starts[s] + j]] for j in range(kept[s])] for s in range(server.B)]


def exps(scale):
    return np.round(np.log2(np.maximum(scale.double().cpu().numpy().T, 2.0 ** R.E_MIN))).astype(np.int64)


@pytest.mark.parametrize("fmt", ["e4m3p", "int8p"])
@pytest.mark.parametrize("how", ["greedy", "target", "draft"])
@pytest.mark.parametrize("n", [9, 40])
def test_accepted_tokens_move_and_the_cache_holds_them(kvq, fmt, how, n):
    """Every walk and every move is the oracle's, bit for bit; in the end the cache holds what the accepted tokens are."""
    server, rng = server_of(kvq, fmt, 3, n, seed=n, how=how, watch=True), np.random.default_rng(n)
    said, times, tally, grown = [[], [], []], [[], [], []], Tally(), 0
    for at, got in enumerate(run_steps(server, rng, STEPS, server.step, tally)):
        for s in range(3):
            said[s] += got[s]
            times[s] += [at] * len(got[s])
        lens, starts = server.lens.tolist(), server.starts.tolist()
        assert lens == [len(x) for x in said]
        rows, table = starts[-1], server.table.cpu().numpy()
        keep, kept = server.keep[:rows].cpu().numpy(), server.kept.cpu().numpy()
        if how != "greedy":
            want = T.verify_runs(server.probs[:rows].cpu().numpy(), None if server.draft is None else server.draft[:rows].cpu().numpy(),
                                 server.tokens[:rows].cpu().numpy(), server.parents[:rows].cpu().numpy(), server.uniform[:rows].cpu().numpy(), starts)
            assert np.array_equal(keep, want[0]) and np.array_equal(kept, want[1]) and server.next.tolist() == want[2].tolist()
        for i, cache in enumerate(server.caches):
            k, v, k_scale, v_scale = server.before[4 * i:4 * i + 4]
            for plane, code, scale, was, was_scale in (("k", cache.k, cache.k_scale, k, k_scale), ("v", cache.v, cache.v_scale, v, v_scale)):
                codes, e = unpack(was.cpu().numpy(), H, fmt, plane), exps(was_scale)
                T.keep_runs(codes, e, keep, kept, starts, lens, table, fmt)
                assert np.array_equal(unpack(code.cpu().numpy(), H, fmt, plane), codes)
                assert np.array_equal(exps(scale), e)
                grown += int((e > exps(was_scale)).sum())
    assert tally.accepted >= 30 and tally.moved >= 12, vars(tally)
    assert n == 9 or tally.across >= 6 and grown >= 6, vars(tally) | dict(grown=grown)
    table, lens = server.table.cpu().numpy(), server.lens.tolist()
    for i, cache in enumerate(server.caches):
        for s in range(3):
            x = server.embed[i][torch.tensor(said[s], device="cuda")]
            k = x[:, H * G:H * G + H].clone()
            kvq.rope_runs(None, k, torch.arange(lens[s], dtype=torch.int32, device="cuda"), server.cos_sin, k_weight=server.weight)
            v = x[:, H * G + H:].double() * 2.0 ** (torch.tensor(times[s], device="cuda") - STEPS)[:, None, None]
            for plane, sc, want in (("k", cache.k_scale, k), ("v", cache.v_scale, v)):
                codes = R.values(unpack(getattr(cache, plane).cpu().numpy(), H, fmt, plane), fmt)
                at = np.arange(lens[s])
                pages = table[s, at // 16]
                step = sc.double().cpu().numpy().T[pages][:, :, None]
                want = want.double().cpu().numpy()
                # rounded when appended and whenever the page's scale grows, under scales of at most the final one: INT8 less than a step of it
                # altogether (1/2 + 1/4 + ..); E4M3 half a step (2^-4 of the value), and half the smallest step (2^-10 of the scale) for each
                # growth, of which a token has at most one for each exponent between -24 and 15
                bound = step if fmt == "int8p" else 2.0 ** -4 * np.abs(want) * 1.01 + 40 * 2.0 ** -10 * step
                assert np.all(np.abs(codes[pages, :, at % 16] * step - want) <= bound)


@pytest.mark.parametrize("n,dtype,how", [(9, torch.bfloat16, "target"), (24, torch.bfloat16, "draft"), (9, torch.float32, "draft")])
def test_a_captured_step_that_moves_repeats_the_eager_one(kvq, n, dtype, how):
    """Two graphs with buffers of their own, replayed in turn beside eager steps."""
    servers = [server_of(kvq, "int8p", 4, n, seed=1, how=how, dtype=dtype) for _ in range(3)]
    runs = [servers[0].step]
    for server in servers[1:]:
        warm = torch.cuda.Stream()
        warm.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(warm):
            server.step()  # of no tokens
        warm.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            server.step()
        runs.append(graph.replay)
    tally = Tally()
    its = [run_steps(s, np.random.default_rng(7), 8, f, tally if s is servers[0] else None) for s, f in zip(servers, runs)]
    for a, b, c in zip(*its):
        assert a == b == c
        used = servers[0].starts[-1].item()
        for other in servers[1:]:
            for x, y in zip(servers[0].caches, other.caches):
                assert all(torch.equal(getattr(x, p), getattr(y, p)) for p in ("k", "v", "k_scale", "v_scale"))
            for name in ("table", "lens", "held", "count", "kept", "next"):
                assert torch.equal(getattr(servers[0], name), getattr(other, name)), name
            assert torch.equal(servers[0].keep[:used], other.keep[:used]) and torch.equal(servers[0].out[:used], other.out[:used])
    assert tally.accepted >= 24 and tally.moved >= 12, vars(tally)


def test_steps_that_move_from_two_threads(kvq):
    cases = [("e4m3p", 2, 30, "draft"), ("int8p", 20, 6, "target")]
    servers, alone = ([server_of(kvq, f, b, n, seed=3, how=how) for f, b, n, how in cases] for _ in range(2))
    faults, barrier, tallies = [], threading.Barrier(2), [Tally(), Tally()]

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                barrier.wait(timeout=30)
                for _ in run_steps(servers[i], np.random.default_rng(i), 10, lambda: servers[i].step(stream), tallies[i]):
                    pass
        except Exception as e:  # noqa: BLE001
            faults.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults, faults
    for i in range(2):
        for _ in run_steps(alone[i], np.random.default_rng(i), 10, alone[i].step):
            pass
        for a, b in zip(servers[i].state(), alone[i].state()):
            assert torch.equal(a, b)
        assert tallies[i].accepted >= 16 and tallies[i].moved >= 8, vars(tallies[i])
