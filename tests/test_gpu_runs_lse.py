"""lse of kvq_attn_runs where value scales are tiny or far apart (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("torch")

import tests.test_gpu_runs as T  # noqa: E402
from tests.runs_cases import FMTS  # noqa: E402
from tests.test_gpu_runs import kvq  # noqa: E402,F401


def tolerance(lse, xa):
    """The exponent e_v of a value scale (-24 .. 15) is part of y = x log2 e + e_v, of the running maximum m and of the sum l of
    2^{y - m + shift - e_v}.  For logits of a few units (larger ones: 2^-17 xa, 128 products) binary32 rounds by half a step, in
    units of log2: shift - m, below 32, 2^-20; e_v + that, below 32, 2^-20; y - m + shift, below 64 where a page's scale is 2^39
    times the one that holds the sum, 2^-19; ex2 2^-22 of the weight; log2 l, below 32, one whole step, 2^-19; less shift, 2^-20; plus
    m, 2^-20 at most.  Together (1 + 1 + 2 + 0.4 + 2 + 1 + 1) 2^-20 = 8.4 x 2^-20, times ln 2 = 5.8 x 2^-20 < 2^-17."""
    return 2.0 ** -17 * xa + 2.0 ** -17 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exps", [(-24, -24), (-20, 2), (-12, -1), (15, 15)])
@pytest.mark.parametrize("new", [[1, 1, 1], [5, 2, 1], [60, 90, 20]])
def test_lse_with_value_scales_in_the_exponent(kvq, monkeypatch, fmt, dtype, exps, new):  # noqa: F811
    monkeypatch.setattr(T, "lse_tolerance", tolerance)
    # keys have the same exponents: queries that keep the logits small
    T.attention_case(kvq, fmt, dtype, [60, 90, 20], new, 4, 5, seed=exps[0] + 30, exps=exps, q_scale=0.01 * 2.0 ** -max(0, exps[1]))
