"""Pins of the oracle's page maps, page-scaled append and causal attention (CPU)."""
import math

import numpy as np
import pytest

from oracle import runs as R
from tests.runs_cases import FMTS, pack, random_codes, starts_of, tables, unpack


def test_map_hands_pages_back_then_out_from_the_top():
    table = np.array([[7, 8, -1], [5, -1, -1], [-1, -1, -1]], dtype=np.int32)
    m = R.map_runs([-1, 3, 17], [20, 15, 0], [1, 2, 3, 0, 0], 3, table, 24)
    # request 0 (2 pages) finished: stack 1 2 3 7 8; request 1 needs one page (8), request 2 two (7, 3)
    assert m["ok"] and m["count"] == 2 and m["stack"].tolist() == [1, 2, 3, 0, 0]
    assert m["table"].tolist() == [[7, 8, -1], [5, 8, -1], [7, 3, -1]]
    assert m["seq_lens"].tolist() == [0, 18, 17] and m["run_starts"].tolist() == [0, 0, 3, 20]
    assert m["slots"][:4].tolist() == [5 * 16 + 15, 8 * 16, 8 * 16 + 1, 7 * 16] and m["slots"][20:].tolist() == [-1] * 4
    assert m["positions"][:4].tolist() == [15, 16, 17, 0]
    m = R.map_runs([-1, 0, 0], [20, 15, 0], [1, 2, 3, 0, 0], 3, table, 0)
    assert m["count"] == 5 and m["stack"].tolist() == [1, 2, 3, 7, 8]
    assert not R.map_runs([0, 0, 97], [20, 15, 0], [1, 2, 3, 0, 0], 3, np.full((3, 8), 4, np.int32), 200)["ok"]


@pytest.mark.parametrize("fmt", FMTS)
def test_page_exponent_is_the_smallest(fmt):
    q = R.QMAX[fmt]
    for e in (-24, -5, 0, 15):
        assert R.page_exponent(q * 2.0 ** e, fmt) == e
        assert R.page_exponent(np.nextafter(q * 2.0 ** e, np.inf), fmt) == min(e + 1, 15)
    assert R.page_exponent(0.0, fmt) == -24 and R.page_exponent(1e30, fmt) == 15


@pytest.mark.parametrize("fmt", FMTS)
def test_append_error_bound_under_growth(fmt):
    """Whatever the order in which a page's scale grows: INT8 within one step of the final scale, E4M3 within half a step
    of the code (2^-4 of the value, or half the smallest subnormal step per growth)."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((16, 1, 128)) * (1.7 ** np.arange(16))[:, None, None]
    codes, exps = np.zeros((1, 1, 16, 128), np.int64), np.zeros((1, 1), np.int64)
    for t in range(16):
        R.append_runs(codes, exps, x[t:t + 1], [0, 1], [t + 1], np.zeros((1, 1), np.int32), fmt)
    step = 2.0 ** int(exps[0, 0])
    assert int(exps[0, 0]) == R.page_exponent(np.abs(x).max(), fmt)
    err = np.abs(R.values(codes[0, 0], fmt) * step - x[:, 0])
    assert np.all(err <= (step if fmt == "int8p" else np.maximum(2.0 ** -4 * np.abs(x[:, 0]), 0) + 2.0 ** -9 * step))


@pytest.mark.parametrize("fmt", FMTS)
def test_attend_one_token_and_uniform_weights(fmt):
    rng = np.random.default_rng(5)
    table, n = tables(rng, [1, 40])
    k, v = random_codes(rng, n, 2, fmt), random_codes(rng, n, 2, fmt)
    e = np.zeros((n, 2), np.int64)
    q = np.zeros((3, 4, 128))
    out, lse, _, _, _ = R.attend(k, e, v, e, q, starts_of([1, 2]), [1, 40], table, 1.0, fmt)
    assert np.array_equal(out[0, 3], R.values(v[table[0, 0], 1, 0], fmt)) and lse[0, 0] == 0.0
    tok = np.concatenate([R.values(v[p, 0], fmt) for p in table[1]])
    np.testing.assert_allclose(out[1, 0], tok[:39].mean(0), rtol=1e-12)
    np.testing.assert_allclose(out[2, 1], tok[:40].mean(0), rtol=1e-12)
    assert abs(lse[2, 0] - math.log(40)) < 1e-12


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("plane", ["k", "v"])
def test_pack_round_trip(fmt, plane):
    c = random_codes(np.random.default_rng(1), 5, 3, fmt)
    assert np.array_equal(unpack(pack(c, fmt, plane), 3, fmt, plane), c)
