"""A step with prompts and trees (GPU): requests with trees first, those with prompts behind them, each kind by its own calls on a slice of the step."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import runs as R  # noqa: E402
from oracle import trees as T  # noqa: E402
from tests.runs_cases import attn_tolerance, random_codes, starts_of, tables  # noqa: E402
from tests.test_gpu_runs import dev, err_word, make_cache  # noqa: E402
from tests.tree_cases import distribution, random_trees  # noqa: E402


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("trees,prompts", [([5, 0, 30], [1100, 3]), ([1, 2], [1]), ([3, 4, 2], [200, 0, 17])])
def test_each_kind_of_run_by_its_own_calls(kvq, dtype, trees, prompts):
    rng = np.random.default_rng(len(trees) + len(prompts))
    H, Hq, V = 2, 8, 40
    at, new = len(trees), trees + prompts
    lens = np.array(new) + rng.integers(0, 60, len(new))
    starts, rows, drafted = starts_of(new), sum(new), sum(trees)
    table, pages = tables(rng, lens)
    ck, cv = (random_codes(rng, pages, H, "e4m3p") for _ in range(2))
    ek, ev = (rng.integers(-9, -6, (pages, H)) for _ in range(2))
    cache = make_cache(kvq, "e4m3p", H, pages, ck, cv, ek, ev)
    parents = np.concatenate([random_trees(rng, trees, 3), np.zeros(rows - drafted, np.int32)])
    q = torch.as_tensor(rng.standard_normal((rows, Hq, 128))).to("cuda", dtype)
    d = dict(starts=dev(starts), lens=dev(lens), table=dev(table), parents=dev(parents))
    words = (max(trees) + 31) // 32
    mask, positions, err = torch.full((rows, words), 7, dtype=torch.int32, device="cuda"), torch.full((rows,), 7, dtype=torch.int32, device="cuda"), err_word()
    out = torch.full_like(q, 7)
    size = max(kvq.attn_tree_workspace_size(at, rows, max(trees), H, Hq, dtype), kvq.attn_runs_workspace_size(len(prompts), rows, max(prompts), H, Hq, dtype))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    first = dict(run_starts=d["starts"][:at + 1], err=err)
    kvq.tree_runs(d["parents"], d["lens"][:at], mask, positions=positions, **first)
    kvq.attn_tree(cache, q, d["lens"][:at], d["table"][:at], mask, out, ws, max_run=max(trees), **first)
    assert torch.all(out[drafted:] == 7) and torch.all(mask[drafted:] == 7) and torch.all(positions[drafted:] == 7)
    kvq.attn_runs(cache, q, d["lens"][at:], d["table"][at:], out, ws, run_starts=d["starts"][at:], max_run=max(prompts), err=err)
    assert err.item() == 0
    want_mask, pos = T.tree_runs(parents[:drafted], starts[:at + 1], lens[:at], words)
    assert np.array_equal(mask[:drafted].cpu().numpy(), want_mask) and np.array_equal(positions[:drafted].cpu().numpy(), pos)
    x = q.double().cpu().numpy()
    a = T.attend_tree(ck, ek, cv, ev, x[:drafted], starts[:at + 1], lens[:at], table[:at], want_mask, 128 ** -0.5, "e4m3p")
    b = R.attend(ck, ek, cv, ev, x[drafted:], starts[at:] - drafted, lens[at:], table[at:], 128 ** -0.5, "e4m3p")
    want, _, pv, xa, low = (np.concatenate(t) for t in zip(a, b))
    off = np.abs(out.double().cpu().numpy() - want) - attn_tolerance(want, pv, xa, low, dtype is torch.bfloat16)
    assert np.all(off <= 0), float(off.max())
    # the trees' paths are verified and kept; the prompts' lengths and pages stay
    p = np.stack([distribution(rng, V) for _ in range(rows)])
    tokens, u = rng.integers(0, V, rows), rng.random((rows, 2)).astype(np.float32)
    keep, kept, following, after = dev(np.full(rows, 7)), dev([7] * at), dev([7] * at), d["lens"].clone()
    was = cache.k.clone()
    kvq.verify_runs(torch.as_tensor(p).cuda(), dev(tokens), d["parents"], torch.as_tensor(u).cuda(), keep, kept, following, seq_lens=after[:at],
                    seq_lens_out=after[:at], **first)
    kvq.keep_runs(cache, after[:at], d["table"][:at], keep, kept, **first)
    assert err.item() == 0
    walk = T.verify_runs(p, None, tokens, parents, u, starts[:at + 1])
    assert keep[:drafted].tolist() == walk[0][:drafted].tolist() and torch.all(keep[drafted:] == 7)
    assert kept.tolist() == walk[1].tolist() and following.tolist() == walk[2].tolist()
    assert after.tolist() == (lens[:at] - np.array(trees) + walk[1]).tolist() + lens[at:].tolist()
    others = np.unique(table[at:][table[at:] >= 0])
    assert torch.equal(cache.k.view(pages, -1)[others], was.view(pages, -1)[others])


@pytest.mark.parametrize("trees,prompts", [([9, 33, 1], [1500, 20]), ([2], [40, 1, 0])])
def test_map_rotation_and_append_take_both(kvq, trees, prompts):
    """One step of both kinds stores what a step of each would have stored: positions are the map's, and the trees' those of tree_runs."""
    rng = np.random.default_rng(len(prompts))
    H, at, new = 2, len(trees), trees + prompts
    before = [int(x) for x in rng.integers(0, 40, len(new))]
    parents = random_trees(rng, trees, 3)
    x = torch.as_tensor(rng.standard_normal((sum(new), 3 * H, 128))).to("cuda", torch.bfloat16)
    angles = torch.arange(1700, device="cuda").double()[:, None] * 1e4 ** (-torch.arange(64, device="cuda").double() / 64)
    table_of_angles = torch.cat([angles.cos(), angles.sin()], 1).float().contiguous()
    weight = torch.as_tensor(1 + 0.1 * rng.standard_normal(128)).to("cuda", torch.float32)

    def step(which, drafted):
        """Requests ``which``, the first ``drafted`` of them with trees -> per request its codes and scales."""
        B, lens0, counts = len(which), [before[s] for s in which], [new[s] for s in which]
        rows = sum(counts)
        first = sum(new[:which[0]])
        mine = x[first:first + rows].clone()
        pages = 4 + sum(-(-(a + b) // 16) for a, b in zip(lens0, counts))
        cache = kvq.PagedCache("int8p", "int8p", H, pages)
        width = max(-(-(a + b) // 16) for a, b in zip(lens0, counts))
        # the context of each request: pages in order, never written
        table = np.full((B, width), -1)
        used = 0
        for s, n in enumerate(lens0):
            table[s, :-(-n // 16)] = np.arange(used, used - (-n // 16))
            used -= -n // 16
        lens, bt, starts, err = dev(lens0), dev(table), dev([0] * (B + 1)), err_word()
        free, count, positions = dev(np.arange(used, pages)), dev([pages - used]), dev([7] * rows)
        kvq.map_runs(dev(counts), lens, free, count, bt, starts, lens, count, max_rows=rows, positions=positions, err=err)
        run = dict(run_starts=starts, err=err)
        if drafted:
            mask = torch.zeros((rows, (max(trees) + 31) // 32), dtype=torch.int32, device="cuda")
            own = dev(np.concatenate([parents, np.zeros(rows - len(parents), np.int32)]))
            kvq.tree_runs(own, lens[:drafted], mask, positions=positions, run_starts=starts[:drafted + 1], err=err)
        kvq.rope_runs(mine[:, :H], mine[:, H:2 * H], positions, table_of_angles, k_weight=weight, **run)
        kvq.append_runs(cache, mine[:, H:2 * H], mine[:, 2 * H:], lens, bt, **run)
        assert err.item() == 0 and lens.tolist() == [a + b for a, b in zip(lens0, counts)]
        t, held = bt.cpu().numpy(), []
        for s in range(B):
            p = torch.as_tensor(t[s, :-(-lens[s].item() // 16)].astype(np.int64), device="cuda")
            held.append([z.view(pages, H, 2048)[p] for z in (cache.k, cache.v)] + [z[:, p] for z in (cache.k_scale, cache.v_scale)])
        return held, positions, mine

    held, positions, rotated = step(list(range(len(new))), at)
    a, pa, ra = step(list(range(at)), at)
    b, pb, rb = step(list(range(at, len(new))), 0)
    assert torch.equal(positions, torch.cat([pa, pb])) and torch.equal(rotated, torch.cat([ra, rb]))
    _, depth = T.tree_runs(parents, starts_of(trees), np.array(before[:at]) + trees, (max(trees) + 31) // 32)
    chain = np.concatenate([np.arange(before[at + i], before[at + i] + n) for i, n in enumerate(prompts)])
    assert positions.tolist() == depth.tolist() + chain.tolist()
    for one, alone in zip(held, a + b):
        assert all(torch.equal(p, q) for p, q in zip(one, alone))
