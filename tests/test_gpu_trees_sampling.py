"""The law of the walk: tokens that come out of verify_runs are distributed as the target says (GPU; the oracle's, CPU).

N independent trees with children drawn from q.  A count of N trials of probability p has a standard deviation of sqrt(N p (1 - p)); every
frequency is held to 6 of them (a chance of 2e-9 for each, and the draws are seeded).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import trees as T  # noqa: E402
from tests.runs_cases import starts_of  # noqa: E402

# Whole 64ths: exact in bf16, and a row's sum is 1.
P = np.array([[32, 19, 3, 10], [6, 13, 19, 26], [45, 7, 6, 6], [16, 16, 16, 16], [3, 3, 38, 20]], np.float32) / 64
Q = np.array([[7, 13, 25, 19], [26, 19, 13, 6], [6, 6, 7, 45], [3, 29, 29, 3], [13, 19, 13, 19]], np.float32) / 64
assert np.all(P.sum(-1) == 1) and np.all(Q.sum(-1) == 1)
TREES = {"two": [-1, 0, 0], "three": [-1, 0, 0, 0], "deep": [-1, 0, 0, 1, 1, 2]}


def draws(rng, parents, n):
    """Trees of n requests: a row's distributions go by its own token (the root's is row 4's), children are draws from them."""
    size = len(parents)
    tokens = np.full((n, size), 4)
    for i in range(1, size):
        cum = np.cumsum(Q.astype(np.float64), -1)[tokens[:, parents[i]]]
        tokens[:, i] = (rng.random(n)[:, None] * cum[:, -1:] > cum).sum(-1)
    return tokens.reshape(-1), rng.random((n * size, 2)).astype(np.float32)


def check(tokens, size, keep, kept, following):
    """The first token after the root is P[4]'s; the second, given the first and where the first was accepted, is the first's row of P."""
    n = len(kept)
    tokens, keep = tokens.reshape(n, size), keep.reshape(n, size)
    path = np.take_along_axis(tokens, np.maximum(keep, 0), 1)
    first = np.where(kept > 1, path[:, 1], following)

    def hold(got, p):
        p = p.astype(np.float64)
        count = np.bincount(got, minlength=4)
        assert np.all(np.abs(count - len(got) * p) <= 6 * np.sqrt(len(got) * p * (1 - p))), (count, len(got) * p)

    hold(first, P[4])
    for x in range(4):
        on = (kept > 1) & (first == x)
        assert on.sum() > 50
        hold(np.where(kept[on] > 2, path[on][:, min(2, size - 1)], following[on]), P[x])


@pytest.mark.parametrize("name", TREES)
@pytest.mark.parametrize("drafts", [True, False])
def test_the_oracles_walk(name, drafts):
    parents = TREES[name]
    n, size = 6000, len(parents)
    tokens, u = draws(np.random.default_rng(size), parents, n)
    keep, kept, following = T.verify_runs(P[tokens], Q[tokens] if drafts else None, tokens, parents * n, u, starts_of([size] * n))
    check(tokens, size, keep, kept, following)


def test_a_walk_that_tries_siblings_against_the_target_alone_is_seen():
    """The planted mistake, in the oracle: after a refusal the next child is tried against p again."""
    parents, n = TREES["three"], 6000
    tokens, u = draws(np.random.default_rng(4), parents, n)
    was = T.residual
    T.residual = lambda p, q, c: was(p, q, np.float32(0))
    try:
        keep, kept, following = T.verify_runs(P[tokens], Q[tokens], tokens, parents * n, u, starts_of([4] * n))
    finally:
        T.residual = was
    with pytest.raises(AssertionError):
        check(tokens, 4, keep, kept, following)


@pytest.mark.gpu
@pytest.mark.parametrize("name", TREES)
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_kernels_walk(name, drafts, dtype):
    import quantized_kv_cache_kvq_gb300 as kvq

    kvq.load()
    parents, calls, batch = TREES[name], 40, 1024
    size = len(parents)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    rng = np.random.default_rng(size)
    out = []
    starts = i32(starts_of([size] * batch))
    for _ in range(calls):
        tokens, u = draws(rng, parents, batch)
        keep, kept, following, err = i32(np.zeros(batch * size)), i32(np.zeros(batch)), i32(np.zeros(batch)), i32([0])
        kvq.verify_runs(torch.as_tensor(P[tokens]).to("cuda", dtype), i32(tokens), i32(parents * batch), torch.as_tensor(u).cuda(), keep, kept, following,
                        draft=torch.as_tensor(Q[tokens]).to("cuda", dtype) if drafts else None, run_starts=starts, err=err)
        assert err.item() == 0
        out.append((tokens, keep.cpu().numpy(), kept.cpu().numpy(), following.cpu().numpy()))
    tokens, keep, kept, following = (np.concatenate(x) for x in zip(*out))
    check(tokens, size, keep, kept, following)
