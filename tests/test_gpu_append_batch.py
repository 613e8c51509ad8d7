"""kvq_append_runs at the largest batch, whose tables leave an SM fewer blocks (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import runs as R  # noqa: E402
from tests.runs_cases import FMTS, random_codes, starts_of, tables  # noqa: E402
from tests.test_gpu_runs import check_cache, dev, err_word, kvq, make_cache  # noqa: E402,F401


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,heads", [(1024, 3), (1023, 1), (600, 5)])
def test_append_of_a_large_batch_equals_the_oracle(kvq, fmt, dtype, batch, heads):  # noqa: F811
    rng = np.random.default_rng(batch)
    old, new = rng.integers(0, 40, batch), rng.integers(0, 30, batch)
    new[rng.integers(batch)] = 200
    lens = old + new
    table, pages = tables(rng, lens)
    ck, cv = random_codes(rng, pages, heads, fmt), random_codes(rng, pages, heads, fmt)
    ek, ev = rng.integers(-9, -2, (pages, heads)), rng.integers(-9, -2, (pages, heads))
    cache = make_cache(kvq, fmt, heads, pages, ck, cv, ek, ev)
    x = torch.as_tensor(rng.standard_normal((int(new.sum()), 2 * heads, 128)) * 2.0 ** rng.integers(-4, 3, (int(new.sum()), 1, 1))).to("cuda", dtype)
    y, starts, err = x.double().cpu().numpy(), starts_of(new), err_word()
    R.append_runs(ck, ek, y[:, :heads], starts, lens, table, fmt)
    R.append_runs(cv, ev, y[:, heads:], starts, lens, table, fmt)
    kvq.append_runs(cache, x[:, :heads], x[:, heads:], dev(lens), dev(table), run_starts=dev(starts), err=err)
    assert err.item() == 0
    check_cache(cache, fmt, heads, ck, cv, ek, ev)
