"""Workspaces of kvq_attn_tree (GPU): one that is large enough for a step is so for every smaller one."""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import trees as T  # noqa: E402
from tests.runs_cases import random_codes, starts_of, tables  # noqa: E402
from tests.test_gpu_runs import dev, err_word, make_cache  # noqa: E402
from tests.tree_cases import random_trees  # noqa: E402


@pytest.fixture(scope="module")
def kvq():
    import quantized_kv_cache_kvq_gb300 as m

    m.load()
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,group", [(1, 1), (8, 4), (4, 7), (2, 8), (128, 1)])
def test_sizes_do_not_fall(kvq, dtype, heads, group):
    """In each of batch, rows and max_run, the others as they are: so in all of them together."""
    axes = [(1, 2, 16, 1000, 1024), (0, 1, 2, 7, 16, 17, 300, 1024, 5000, 65536), (0, 1, 2, 3, 4, 5, 8, 9, 16, 17, 64, 1000, 1024)]
    size = {x: kvq.attn_tree_workspace_size(*x, heads, heads * group, dtype) for x in itertools.product(*axes)}
    for at, axis in enumerate(axes):
        for a, b in zip(axis, axis[1:]):
            for x in size:
                if x[at] == a:
                    assert 0 < size[x] <= size[x[:at] + (b,) + x[at + 1:]], (x, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_workspace_of_the_largest_step_serves_smaller_ones(kvq, dtype):
    """A server of 16 requests, 8 and 32 heads and trees of up to 64 tokens, whose next step has small trees, or fewer requests."""
    H, Hq, B, n = 8, 32, 16, 64
    rng = np.random.default_rng(0)
    lens = rng.integers(70, 200, B)
    table, pages = tables(rng, lens)
    codes, e = random_codes(rng, pages, H, "int8p"), rng.integers(-8, -4, (pages, H))
    cache = make_cache(kvq, "int8p", H, pages, codes, codes, e, e)
    rows = B * n
    q = torch.randn((rows, Hq, 128), device="cuda").to(dtype)
    large = torch.empty(kvq.attn_tree_workspace_size(B, rows, n, H, Hq, dtype), dtype=torch.uint8, device="cuda")
    for batch, most, held in ((16, 64, rows), (16, 4, rows), (16, 4, 64), (16, 1, 16), (3, 2, rows), (1, 64, 64), (2, 17, 40)):
        new = rng.integers(1, most + 1, batch) if held > batch * most - 1 else np.full(batch, held // batch)
        starts = starts_of(new)
        mask, _ = T.tree_runs(random_trees(rng, new, 3), starts, lens[:batch], (most + 31) // 32)
        mask = np.concatenate([mask, np.zeros((held - len(mask), mask.shape[1]), np.int32)])
        own = torch.empty(kvq.attn_tree_workspace_size(batch, held, most, H, Hq, dtype), dtype=torch.uint8, device="cuda")
        outs = []
        for ws in (own, large):
            out, err = torch.zeros_like(q[:held]), err_word()
            kvq.attn_tree(cache, q[:held], dev(lens[:batch]), dev(table[:batch]), dev(mask), out, ws, run_starts=dev(starts), max_run=most, err=err)
            assert err.item() == 0
            outs.append(out)
        assert own.nbytes <= large.nbytes and torch.equal(*outs)
        assert torch.all(torch.any(outs[0][:int(starts[-1])] != 0, -1)) and torch.all(outs[0][int(starts[-1]):] == 0)
