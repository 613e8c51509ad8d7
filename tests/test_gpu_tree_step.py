"""Speculative steps as a server runs them (GPU): map -> masks -> rotation -> append -> attention -> verification -> kept path, and on.

What the cache holds after steps with trees is what a server that appends the accepted tokens one by one would have stored, to the
rounding of the page scales; the steps run eagerly, as one captured graph, and from two threads, with the same bits.
"""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import runs as R  # noqa: E402
from tests.runs_cases import starts_of, unpack  # noqa: E402
from tests.tree_cases import random_tree  # noqa: E402

H, G, V, LAYERS = 2, 2, 64, 3


class Server:
    """A toy model over a table of embeddings: what a step computes depends on the cache through the attention of its last layer."""

    def __init__(self, kvq, fmt, batch, n, seed, dtype=torch.bfloat16, greedy=False):
        self.kvq, self.fmt, self.B, self.n, self.greedy = kvq, fmt, batch, n, greedy
        g = torch.Generator(device="cuda").manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.rows = batch * n + 5
        pages = batch * 40
        self.caches = [kvq.PagedCache(fmt, fmt, H, pages, layer=i) for i in range(LAYERS)]
        self.embed = torch.randn((LAYERS, V, H * G + 2 * H, 128), generator=g, device="cuda").to(dtype)
        self.head = torch.randn((H * G * 128, V), generator=g, device="cuda") * 0.15
        theta = 1e6 ** (-torch.arange(64, device="cuda").double() / 64)
        a = torch.arange(700, device="cuda").double()[:, None] * theta
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
        self.weight = 1 + 0.1 * torch.randn(128, generator=g, device="cuda")
        self.free, self.count = torch.arange(pages, **i32), torch.tensor([pages], **i32)
        self.table, self.held = torch.full((batch, 40), -1, **i32), torch.zeros(batch, **i32)
        self.lens, self.starts = torch.zeros(batch, **i32), torch.zeros(batch + 1, **i32)
        self.new = torch.zeros(batch, **i32)
        self.tokens, self.parents = torch.zeros(self.rows, **i32), torch.zeros(self.rows, **i32)
        self.uniform = torch.zeros((self.rows, 2), device="cuda")
        self.mask, self.positions = torch.zeros((self.rows, (n + 31) // 32), **i32), torch.zeros(self.rows, **i32)
        self.out = torch.zeros((self.rows, H * G, 128), dtype=dtype, device="cuda")
        self.ws = torch.empty(kvq.attn_tree_workspace_size(batch, self.rows, n, H, H * G, dtype), dtype=torch.uint8, device="cuda")
        self.keep, self.kept, self.next = torch.zeros(self.rows, **i32), torch.zeros(batch, **i32), torch.zeros(batch, **i32)
        self.err = torch.zeros(1, **i32)
        self.fused = torch.zeros((LAYERS, self.rows, H * G + 2 * H, 128), dtype=dtype, device="cuda")

    def feed(self, trees, tokens, uniform):
        """The drafts of a step, in place (a captured step reads them here)."""
        self.new.copy_(torch.tensor([len(t) for t in trees], dtype=torch.int32))
        flat = [p for t in trees for p in t]
        pad = lambda x: torch.tensor(list(x) + [0] * (self.rows - len(x)), dtype=torch.int32)  # noqa: E731
        self.parents.copy_(pad(flat))
        self.tokens.copy_(pad(tokens))
        self.uniform.copy_(uniform)

    def step(self, stream=None):
        kvq, run = self.kvq, dict(run_starts=self.starts, err=self.err, stream=stream)
        kvq.map_runs(self.new, self.lens, self.free, self.count, self.table, self.starts, self.lens, self.count, held_pages=self.held,
                     max_rows=self.rows, err=self.err, stream=stream)
        kvq.tree_runs(self.parents, self.lens, self.mask, positions=self.positions, **run)
        for i, cache in enumerate(self.caches):
            x = self.fused[i]
            x.copy_(self.embed[i][self.tokens.long()])
            q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
            kvq.rope_runs(q, k, self.positions, self.cos_sin, q_weight=self.weight, k_weight=self.weight, **run)
            kvq.append_runs(cache, k, v, self.lens, self.table, **run)
            kvq.attn_tree(cache, q, self.lens, self.table, self.mask, self.out, self.ws, max_run=self.n, **run)
        logits = self.out.float().view(self.rows, -1) @ self.head
        self.probs = torch.softmax(logits, -1)
        kvq.verify_runs(logits if self.greedy else self.probs, self.tokens, self.parents, None if self.greedy else self.uniform, self.keep, self.kept,
                        self.next, seq_lens=self.lens, seq_lens_out=self.lens, **run)
        kvq.keep_runs(self.caches, self.lens, self.table, self.keep, self.kept, **run)

    def state(self):
        return [t.clone() for c in self.caches for t in (c.k, c.v, c.k_scale, c.v_scale)] + [
            t.clone() for t in (self.table, self.lens, self.held, self.free, self.count, self.keep, self.kept, self.next, self.out, self.err)]


def drafts(rng, batch, n, last):
    """Trees of up to n rows whose roots are the tokens chosen last."""
    trees = [random_tree(rng, int(rng.integers(1, n + 1)), 3) for _ in range(batch)]
    tokens = [t for s, tree in enumerate(trees) for t in [int(last[s])] + rng.integers(0, V, len(tree) - 1).tolist()]
    return trees, tokens


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


def steps(server, rng, count, run):
    """Feeds and runs ``count`` steps; yields what was accepted in each: a list of tokens for each request."""
    last = rng.integers(0, V, server.B)
    for _ in range(count):
        trees, tokens = drafts(rng, server.B, server.n, last)
        server.feed(trees, tokens, torch.as_tensor(rng.random((server.rows, 2)).astype(np.float32)))
        run()
        torch.cuda.synchronize()
        assert server.err.item() == 0
        starts = starts_of([len(t) for t in trees])
        kept, keep = server.kept.tolist(), server.keep.tolist()
        last = np.array(server.next.tolist())
        yield [[tokens[starts[s] + keep[starts[s] + j]] for j in range(kept[s])] for s in range(server.B)]


@pytest.mark.parametrize("fmt", ["e4m3p", "int8p"])
@pytest.mark.parametrize("n", [3, 9, 40])
def test_the_cache_holds_the_accepted_tokens(kvq, fmt, n):
    server = Server(kvq, fmt, 3, n, seed=n, greedy=True)
    rng = np.random.default_rng(n)
    said = [[], [], []]
    total = 0
    for got in steps(server, rng, 25, server.step):
        for s in range(3):
            said[s] += got[s]
            total += len(got[s])
        assert server.lens.tolist() == [len(x) for x in said]
    table, lens = server.table.cpu().numpy(), server.lens.tolist()
    used = table[table >= 0]
    assert len(set(used.tolist()) | set(server.free[:server.count.item()].tolist())) == 120
    assert all(server.held[s].item() >= -(-lens[s] // 16) for s in range(3))
    for i, cache in enumerate(server.caches):
        for s in range(3):
            tok = torch.tensor(said[s], device="cuda")
            x = server.embed[i][tok]
            k = x[:, H * G:H * G + H].clone()
            kvq.rope_runs(None, k, torch.arange(lens[s], dtype=torch.int32, device="cuda"), server.cos_sin, k_weight=server.weight)
            for plane, sc, want in (("k", cache.k_scale, k), ("v", cache.v_scale, x[:, H * G + H:])):
                codes = R.values(unpack(getattr(cache, plane).cpu().numpy(), H, fmt, plane), fmt)
                scale = sc.double().cpu().numpy()
                at = np.arange(lens[s])
                pages = table[s, at // 16]
                held = codes[pages, :, at % 16] * scale.T[pages][:, :, None]
                want = want.double().cpu().numpy()
                # a code is rounded when it is appended and whenever its page's scale grows, under scales of at most the final one:
                # INT8 less than one step of it altogether (1/2 + 1/4 + ..); E4M3 half a step (2^-4), and half the smallest
                # step (2^-10 of the scale) for each of at most 16 growths
                step = scale.T[pages][:, :, None]
                bound = step if fmt == "int8p" else 2.0 ** -4 * np.abs(want) * 1.01 + 2.0 ** -6 * step
                assert np.all(np.abs(held - want) <= bound)


@pytest.mark.parametrize("n,dtype", [(4, torch.bfloat16), (24, torch.bfloat16), (6, torch.float32)])
def test_a_captured_step_repeats_the_eager_one(kvq, n, dtype):
    """One graph for every step, whatever the drafts; two captured graphs with workspaces of their own, replayed in turn."""
    eager, one, two = (Server(kvq, "int8p", 4, n, seed=1, dtype=dtype) for _ in range(3))
    rngs = [np.random.default_rng(7) for _ in range(3)]
    graphs = []
    for server in (one, two):
        warm = torch.cuda.Stream()
        with torch.cuda.stream(warm):
            server.step()  # of no tokens: nothing is appended or kept
        warm.synchronize()
        assert server.lens.tolist() == [0] * 4
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            server.step()
        graphs.append(graph)
    its = [steps(s, r, 8, f) for s, r, f in zip((eager, one, two), rngs, (eager.step, graphs[0].replay, graphs[1].replay))]
    for a, b, c in zip(*its):
        assert a == b == c
        want = eager.state()
        for server in (one, two):
            got = server.state()
            used = server.starts[-1].item()
            got[-2], w = got[-2][:used], want[-2][:used]
            assert torch.equal(got[-2], w)
            assert all(torch.equal(x, y) for i, (x, y) in enumerate(zip(got, want)) if i not in (len(want) - 2, len(want) - 5))
            assert torch.equal(got[-5][:used], want[-5][:used])


def test_steps_from_two_threads(kvq):
    servers = [Server(kvq, "e4m3p", b, n, seed=3) for b, n in ((2, 30), (40, 3))]
    alone = [Server(kvq, "e4m3p", b, n, seed=3) for b, n in ((2, 30), (40, 3))]
    faults, barrier = [], threading.Barrier(2)

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                barrier.wait(timeout=30)
                for _ in steps(servers[i], np.random.default_rng(i), 10, lambda: servers[i].step(stream)):
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
        for _ in steps(alone[i], np.random.default_rng(i), 10, alone[i].step):
            pass
        for a, b in zip(servers[i].state(), alone[i].state()):
            assert torch.equal(a, b)
