"""Trees of drafted tokens at the limits (GPU): caches past 4 GB, queries that are no numbers, rows of different alignment, other streams."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import trees as T  # noqa: E402
from tests.runs_cases import random_codes, starts_of, tables  # noqa: E402
from tests.test_gpu_runs import dev, err_word, make_cache  # noqa: E402
from tests.tree_cases import distribution, random_trees  # noqa: E402


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


def attn(kvq, cache, q, lens, table, mask, starts, max_run):
    rows, Hq, _ = q.shape
    out, lse, err = torch.zeros_like(q), torch.zeros((rows, Hq), device="cuda"), err_word()
    ws = torch.empty(kvq.attn_tree_workspace_size(len(lens), rows, max_run, cache.num_kv_heads, Hq, q.dtype), dtype=torch.uint8, device="cuda")
    kvq.attn_tree(cache, q, dev(lens), dev(table), dev(mask), out, ws, run_starts=dev(starts), max_run=max_run, lse=lse, err=err)
    assert err.item() == 0
    return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_past_4_gb(kvq, dtype):
    """The same tokens in a small cache and on the last pages of a large one: attention and kept paths give the same bits."""
    rng = np.random.default_rng(0)
    H, new, lens = 8, [30, 7], [100, 61]
    table, pages = tables(rng, lens)
    ck, cv = random_codes(rng, pages, H, "int8p"), random_codes(rng, pages, H, "int8p")
    ek, ev = rng.integers(-9, -4, (pages, H)), rng.integers(-9, -4, (pages, H))
    small = make_cache(kvq, "int8p", H, pages, ck, cv, ek, ev)
    total = (1 << 32) // (2048 * H) + 1000  # 4 GB of keys, and more
    big = kvq.PagedCache("int8p", "int8p", H, total)
    shift = total - pages
    big.k[shift * H:], big.v[shift * H:] = small.k, small.v
    big.k_scale[:, shift:], big.v_scale[:, shift:] = small.k_scale, small.v_scale
    far = np.where(table >= 0, table + shift, -1)
    starts = starts_of(new)
    mask, _ = T.tree_runs(random_trees(rng, new, 3), starts, lens, 1)
    q = torch.randn((37, 2 * H, 128), device="cuda").to(dtype)
    for x, y in zip(attn(kvq, small, q, lens, table, mask, starts, 30), attn(kvq, big, q, lens, far, mask, starts, 30)):
        assert torch.equal(x, y)
    keep = np.full(37, -1)
    keep[:3], keep[30:32] = [0, 5, 22], [0, 4]
    for cache, t in ((small, table), (big, far)):
        err = err_word()
        kvq.keep_runs(cache, dev([73, 56]), dev(t), dev(keep), dev([3, 2]), run_starts=dev(starts), err=err)
        assert err.item() == 0
    assert torch.equal(big.k[shift * H:], small.k) and torch.equal(big.v[shift * H:], small.v)
    assert torch.equal(big.k_scale[:, shift:], small.k_scale) and torch.equal(big.v_scale[:, shift:], small.v_scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,bad", [(3, 1), (40, 7), (40, 39)])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_query_that_is_no_number_stays_alone(kvq, dtype, n, bad, what):
    rng = np.random.default_rng(n)
    lens, new = [300, n + 1], [n, n]
    table, pages = tables(rng, lens)
    codes, e = random_codes(rng, pages, 1, "e4m3p"), rng.integers(-8, -4, (pages, 1))
    cache = make_cache(kvq, "e4m3p", 1, pages, codes, codes, e, e)
    mask, _ = T.tree_runs(random_trees(rng, new, 3), starts_of(new), lens, 2)
    q = torch.randn((2 * n, 4, 128), device="cuda").to(dtype)
    want, want_lse = attn(kvq, cache, q, lens, table, mask, starts_of(new), n)
    q[bad, 2, 50] = what
    out, lse = attn(kvq, cache, q, lens, table, mask, starts_of(new), n)
    assert torch.all(torch.isnan(out[bad, 2])) and torch.isnan(lse[bad, 2])
    out[bad, 2], lse[bad, 2] = want[bad, 2], want_lse[bad, 2]
    # the rows of a unit move their maxima together: the same values, not always the same bits
    torch.testing.assert_close(out.float(), want.float(), rtol=2e-2 if dtype is torch.bfloat16 else 1e-5, atol=1e-2 if dtype is torch.bfloat16 else 1e-5)
    torch.testing.assert_close(lse, want_lse, rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("first,second", [(0, 1), (1, 0), (3, 2), (8, 5)])
def test_target_and_draft_of_different_alignment(kvq, dtype, first, second):
    rng = np.random.default_rng(first)
    V, n = 1031, 12
    parents, starts = random_trees(rng, [n], 3), [0, n]
    wide = [torch.full((n, V + 16), 0.5, dtype=dtype, device="cuda") for _ in range(2)]
    held = []
    for w, at in zip(wide, (first, second)):
        w[:, at:at + V] = torch.as_tensor(np.stack([distribution(rng, V, 1.0) for _ in range(n)])).to("cuda", dtype)
        held.append(w[:, at:at + V])
    p, q = (t.float().cpu().numpy() for t in held)
    tokens = np.array([0] + [int(rng.choice(V, p=q[parents[i]].astype(np.float64) / q[parents[i]].astype(np.float64).sum())) for i in range(1, n)])
    u = rng.random((n, 2)).astype(np.float32)
    want = T.verify_runs(p, q, tokens, parents, u, starts)
    keep, kept, following, err = dev([7] * n), dev([7]), dev([7]), err_word()
    kvq.verify_runs(held[0], dev(tokens), dev(parents), dev(u, torch.float32), keep, kept, following, draft=held[1], run_starts=dev(starts), err=err)
    assert err.item() == 0 and keep.tolist() == want[0].tolist() and kept.tolist() == want[1].tolist() and following.tolist() == want[2].tolist()


def test_calls_on_a_stream_of_their_own(kvq):
    """Inputs written on a stream, the calls on it too, while the default stream is busy with something else."""
    rng = np.random.default_rng(5)
    ns = [40, 33]
    parents, starts, lens = random_trees(rng, ns, 3), starts_of(ns), [90, 33]
    want, pos = T.tree_runs(parents, starts, lens, 2)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    with torch.cuda.stream(stream):
        p = dev(parents)
        mask, positions = torch.zeros((73, 2), dtype=torch.int32, device="cuda"), torch.zeros(73, dtype=torch.int32, device="cuda")
        kvq.tree_runs(p, dev(lens), mask, positions=positions, run_starts=dev(starts))
        x = torch.randn((73, 3, 128), device="cuda")
        y = torch.zeros_like(x)
        cs = torch.randn((100, 128), device="cuda")
        kvq.rope_runs(x, None, positions, cs, q_out=y)
    stream.synchronize()
    assert np.array_equal(mask.cpu().numpy(), want) and np.array_equal(positions.cpu().numpy(), pos)
    exact = T.rope(x.double().cpu().numpy(), None, 0.0, pos, cs.double().cpu().numpy())
    assert np.allclose(y.cpu().numpy(), exact, rtol=0, atol=2.0 ** -22 * 100)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_largest_tree_and_the_largest_batch(kvq, dtype):
    """1024 rows in one run; 1024 runs: the same rows one by one through attn_runs (a chain) give the same values."""
    rng = np.random.default_rng(6)
    for new, lens in (([1024], [1030]), ([2] * 1024, list(rng.integers(2, 60, 1024)))):
        table, pages = tables(rng, lens)
        codes, e = random_codes(rng, pages, 1, "int8p"), rng.integers(-8, -4, (pages, 1))
        cache = make_cache(kvq, "int8p", 1, pages, codes, codes, e, e)
        rows, starts = sum(new), starts_of(new)
        parents = dev(np.concatenate([np.arange(n) - 1 for n in new]))
        mask = torch.zeros((rows, (max(new) + 31) // 32), dtype=torch.int32, device="cuda")
        kvq.tree_runs(parents, dev(lens), mask, run_starts=dev(starts))
        q = torch.randn((rows, 8, 128), device="cuda").to(dtype)
        out, _ = attn(kvq, cache, q, lens, table, mask.cpu().numpy(), starts, max(new))
        want = torch.zeros_like(q)
        ws = torch.empty(kvq.attn_runs_workspace_size(len(new), rows, max(new), 1, 8, dtype), dtype=torch.uint8, device="cuda")
        kvq.attn_runs(cache, q, dev(lens), dev(table), want, ws, run_starts=dev(starts), max_run=max(new))
        torch.testing.assert_close(out.float(), want.float(), rtol=2e-2 if dtype is torch.bfloat16 else 1e-4, atol=1e-2 if dtype is torch.bfloat16 else 1e-4)


def test_empty_runs_and_no_rows(kvq):
    """Nothing to keep: the outputs say so."""
    kept, following, lens = dev([7] * 3), dev([7] * 3), dev([4, 0, 9])
    none = torch.zeros((0,), dtype=torch.int32, device="cuda")
    kvq.verify_runs(torch.zeros((0, 50), device="cuda"), none, none, None, none, kept, following, seq_lens=lens, seq_lens_out=lens, run_starts=dev([0] * 4))
    assert kept.tolist() == [0] * 3 and following.tolist() == [-1] * 3 and lens.tolist() == [4, 0, 9]
    cache = kvq.PagedCache("int8p", "int8p", 1, 2)
    kvq.keep_runs([], lens, dev([[0], [0], [0]]), none, kept, run_starts=dev([0] * 4))
    kvq.keep_runs(cache, lens, dev([[0], [0], [0]]), none, kept, run_starts=dev([0] * 4))
    kvq.rope_runs(torch.zeros((0, 2, 128), device="cuda"), None, none, torch.zeros((1, 128), device="cuda"))
