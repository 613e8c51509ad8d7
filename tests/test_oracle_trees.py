"""Pins of the oracle's trees: masks, rotation, attention, verification and the kept path (CPU)."""
import itertools
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import runs as R
from oracle import trees as T
from tests.runs_cases import FMTS, random_codes, starts_of, tables
from tests.tree_cases import distribution, random_trees


def test_masks_and_positions_of_a_small_tree():
    mask, pos = T.tree_runs([-1, 0, 0, 1, -1], [0, 4, 5], [10, 3], 1)
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b1] and pos.tolist() == [6, 7, 7, 8, 2]
    mask, pos = T.tree_runs([-1] + list(range(39)), [0, 40], [40], 2)
    assert mask[39].tolist() == [-1, 255] and pos.tolist() == list(range(40))


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    theta = 1e6 ** (-np.arange(64) / 64)
    cs = np.concatenate([np.cos(np.arange(50)[:, None] * theta), np.sin(np.arange(50)[:, None] * theta)], 1)
    x, y = rng.standard_normal((2, 1, 1, 128))
    at = lambda v, p: T.rope(v, None, 0.0, np.array([p]), cs)[0, 0]  # noqa: E731
    np.testing.assert_allclose(np.linalg.norm(at(x, 31)), np.linalg.norm(x), rtol=1e-12)
    np.testing.assert_allclose(at(x, 12) @ at(y, 5), at(x, 47) @ at(y, 40), rtol=1e-10)
    n = T.rope(x * 1e3, np.full(128, 2.0), 0.0, np.array([0]), cs)
    np.testing.assert_allclose(np.sqrt((n * n).mean()), 2.0, rtol=1e-12)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_chain_is_causal(fmt):
    rng = np.random.default_rng(1)
    new, lens = [5, 0, 20, 1], [12, 3, 20, 40]
    table, n = tables(rng, lens)
    ck, cv = random_codes(rng, n, 2, fmt), random_codes(rng, n, 2, fmt)
    e = rng.integers(-7, -3, (n, 2))
    q = rng.standard_normal((26, 4, 128))
    mask, _ = T.tree_runs(random_trees(rng, new, 1), starts_of(new), lens, 1)
    got = T.attend_tree(ck, e, cv, e, q, starts_of(new), lens, table, mask, 0.1, fmt)
    want = R.attend(ck, e, cv, e, q, starts_of(new), lens, table, 0.1, fmt)
    for x, y in zip(got, want):
        np.testing.assert_allclose(x, y, rtol=1e-12, equal_nan=True)


def naive_residuals(p, q, k):
    """p_0 .. p_k of recursive rejection, each normalised: p_{j+1} = max(p_j - q, 0) / sum."""
    out = [[x / sum(p) for x in p]]
    for _ in range(k):
        r = [max(x - y, Fraction(0)) for x, y in zip(out[-1], q)]
        if sum(r) == 0:
            break
        out.append([x / sum(r) for x in r])
    return out


def test_residuals_have_the_closed_form():
    """max(p - c q, 0) / Z with c += Z is the recursion, in exact arithmetic."""
    rng = np.random.default_rng(2)
    for _ in range(20):
        p = [Fraction(int(x) + 1, 1000) for x in rng.integers(0, 200, 9)]
        q = [Fraction(int(x) + 1, 1000) for x in rng.integers(0, 200, 9)]
        p, q = [x / sum(p) for x in p], [x / sum(q) for x in q]
        c, z = Fraction(0), sum(p)
        for want in naive_residuals(p, q, 4):
            assert [max(x - c * y, Fraction(0)) / z for x, y in zip(p, q)] == want
            c += z
            z = sum(max(x - c * y, Fraction(0)) for x, y in zip(p, q))
            if z == 0:
                break


def test_the_first_token_has_the_targets_distribution():
    """Over all pairs of drafted children and a fine grid of random numbers, the token after the root is distributed as p: the
    probability of each is the integral of the acceptance steps, here counted on a grid of 64 x 64 x 64 numbers."""
    rng = np.random.default_rng(3)
    V, grid = 3, 64
    p, q = distribution(rng, V, 1.0), distribution(rng, V, 1.0)
    u = (np.arange(grid) + 0.5) / grid
    got = np.zeros(V)
    for x, y in itertools.product(range(V), repeat=2):
        weight = float(q[x]) * float(q[y]) / grid ** 3
        z0 = float(p.sum())
        first = u * float(q[x]) * z0 < float(p[x])
        got[x] += weight * grid * grid * first.sum()
        r = T.residual(p, q, np.float32(z0))
        second = u * float(q[y]) * float(r.sum()) < float(r[y])
        refused = (~first).sum()
        got[y] += weight * grid * refused * second.sum()
        r2 = T.residual(p, q, np.float32(z0 + float(r.sum())))
        cum = np.cumsum(r2 / r2.sum()) if r2.sum() else np.ones(V)
        for t in np.searchsorted(cum, u, side="right"):
            got[min(t, V - 1)] += weight * refused * (~second).sum()
    # each of the three thresholds is off by at most one of 64 numbers
    np.testing.assert_allclose(got, p, atol=3 / grid)


def walk(rng, how, V=40):
    ns = [1, 0, 7, 30, 2]
    rows = sum(ns)
    parents = random_trees(rng, ns, 3)
    target = np.stack([distribution(rng, V) for _ in range(rows)])
    draft = np.stack([distribution(rng, V) for _ in range(rows)]) if how == "draft" else None
    tokens = rng.integers(0, V, rows)
    uniform = None if how == "greedy" else rng.random((rows, 2)).astype(np.float32)
    return T.verify_runs(target, draft, tokens, parents, uniform, starts_of(ns)), (ns, parents, tokens, target, uniform)


@pytest.mark.parametrize("how", ["greedy", "target", "draft"])
def test_a_path_goes_from_parent_to_child(how):
    for seed in range(10):
        (keep, kept, last), (ns, parents, tokens, target, _) = walk(np.random.default_rng(seed), how)
        starts = starts_of(ns)
        assert kept[1] == 0 and last[1] == -1
        for s, n in enumerate(ns):
            path = keep[starts[s]:starts[s] + kept[s]].tolist()
            assert path[:1] == [0] * min(n, 1) and np.all(keep[starts[s] + kept[s]:starts[s + 1]] == -1)
            for a, b in zip(path, path[1:]):
                assert parents[starts[s] + b] == a
                if how == "greedy":
                    assert tokens[starts[s] + b] == np.argmax(target[starts[s] + a])
            assert n == 0 or 0 <= last[s] < 40


def test_equal_distributions_accept_the_first_child():
    """q = p: u q < p whatever the random number; and a child with q = 0 and p > 0 is always accepted."""
    p = distribution(np.random.default_rng(4), 50)
    u = np.array([[0, 0.5], [np.nextafter(np.float32(1), np.float32(0)), 0.5]], np.float32)
    keep, kept, _ = T.verify_runs([p, p], [p, p], [0, 7], [-1, 0], u, [0, 2])
    assert kept.tolist() == [2]
    q = p.copy()
    q[7] = 0
    assert T.verify_runs([p, p], [q, q], [0, 7], [-1, 0], u, [0, 2])[1].tolist() == [2]


def test_drawing_takes_the_lowest_token_past_the_threshold():
    w = [0, 3, 0, 5, 2]
    assert [T._draw(w, u / 10) for u in range(10)] == [1] * 3 + [3] * 5 + [4] * 2
    assert T._draw(w, 0.0) == 1 and T._draw(w, 1.0) == 4 and T._draw(w, math.nextafter(1.0, 0.0)) == 4


@pytest.mark.parametrize("fmt", FMTS)
def test_kept_tokens_hold_their_values(fmt):
    """After the move every kept token stands for what it stood for, exactly where its page's scale did not grow and within half a
    step of the new scale elsewhere; other requests' pages are as they were."""
    rng = np.random.default_rng(5)
    new, before = [20, 3, 0, 40], [13, 16, 5, 0]
    after = np.array(before) + new
    table, n = tables(rng, after)
    codes, exps = random_codes(rng, n, 2, fmt), rng.integers(-9, -3, (n, 2))
    paths = [[0, 4, 9, 17], [0, 1, 2], [], list(range(0, 40, 2))]
    keep = np.full(sum(new), -1)
    for s, p in enumerate(paths):
        keep[starts_of(new)[s]:starts_of(new)[s] + len(p)] = p
    kept = np.array([len(p) for p in paths])
    was, had = codes.copy(), exps.copy()
    T.keep_runs(codes, exps, keep, kept, starts_of(new), np.array(before) + kept, table, fmt)
    value = lambda c, e, s, pos: R.values(c[table[s, pos // 16], :, pos % 16], fmt) * 2.0 ** e[table[s, pos // 16]][:, None]  # noqa: E731
    for s, path in enumerate(paths):
        for pos in range(before[s] + len(path)):
            src = pos if pos < before[s] else before[s] + path[pos - before[s]]
            a, b = value(was, had, s, src), value(codes, exps, s, pos)
            step = 2.0 ** exps[table[s, pos // 16]][:, None]
            half = 0.5 * step if fmt == "int8p" else np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * step)
            same = (had[table[s, src // 16]] == exps[table[s, pos // 16]])[:, None]
            assert np.all(np.abs(a - b) <= np.where(same, 0, half))
    for s in (1, 2):
        for p in table[s, :-(-after[s] // 16)]:
            assert np.array_equal(was[p], codes[p]) and np.array_equal(had[p], exps[p])
